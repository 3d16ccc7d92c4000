"""bf16 products grouped by expert against a float64 product on the CPU.

Tolerance: the kernel forms the exact products of bf16 values and adds them
in fp32.  Whatever the order, each of at most k + 1 additions is off by at
most one fp32 step (2^-23, truncation allowed for) of a partial sum that the
sum of magnitudes S bounds: e = (k + 1) 2^-23 S.  A bf16 result adds half a
bf16 step (8 bits), 2^-8 of the value."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu

# (group sizes, N, K): single rows, empty groups, tile edges (128, 256) and one past them,
# contractions below, at and past a stage of 64, one group, more groups than rows
CASES = [
    ([1], 8, 8),
    ([1, 0, 3, 0], 16, 64),
    ([0, 5, 0, 130, 1], 136, 72),
    ([160, 0, 96, 256], 128, 256),
    ([127, 128, 129], 264, 520),
    ([255, 257, 0, 2], 248, 200),
    ([700], 520, 1032),
    ([0, 0, 64], 72, 56),
    ([3] * 40, 40, 136),
]
# at most 8 rows a group on average: blocks of 16 rows that end in a group, contractions that
# end inside a piece of a wave (128), columns that end inside 16
FEW = [([16], 24, 1032), ([17, 0, 1], 40, 4104), ([0, 33, 15, 2, 0, 0, 0, 0], 264, 136), ([1] * 9 + [0] * 300, 16, 8),
       ([0, 0, 48], 8, 2056)]
# every workgroup of the large-tile launch runs several tiles (full output checked)
LARGE = [([1500, 0, 33, 2600, 900, 1, 511, 2047], 1288, 328)]


def _bf16(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16()


def _setup(sizes):
    ends = np.concatenate([[0], np.cumsum(sizes)])
    return ends.tolist(), torch.tensor(ends, dtype=torch.int32, device="cuda")


def _strided(t, extra, at=0):
    """The same values as a slice of a wider tensor whose other columns are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype)
    wide[:, at:at + t.shape[1]] = t
    return wide.cuda()[:, at:at + t.shape[1]]


def _check(got, ref, mag, k, bf16):
    got, e = got.double().cpu(), (k + 1) * 2.0 ** -23 * mag
    tol = e + (2.0 ** -8 * (ref.abs() + e) if bf16 else 2.0 ** -23 * ref.abs())
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / tol.clamp_min(1e-300)).max()))
    assert not got.isnan().any()


def _products(ends, a, b):
    """Per group a[g rows] @ b[g], with the sums of magnitudes (float64)."""
    parts = [(a[s:e].double() @ b[g].double(), a[s:e].double().abs() @ b[g].double().abs())
             for g, (s, e) in enumerate(zip(ends, ends[1:]))]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


@pytest.mark.parametrize("sizes,N,K", CASES + FEW + LARGE)
@pytest.mark.parametrize("pad", [0, 24])
def test_forward(sizes, N, K, pad):
    ends, off = _setup(sizes)
    x, w = _bf16((ends[-1], K), 1), _bf16((len(sizes), N, K), 2)
    ref, mag = _products(ends, x, w.transpose(1, 2))
    out = torch.full((ends[-1], N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mx.mx_grouped_gemm_bf16(_strided(x, pad, 8 if pad else 0), w.cuda(), off, out=out[:, :N])
    _check(got, ref, mag, K, True)
    assert (out[:, N:] == 7.0).all()


@pytest.mark.parametrize("sizes,N,K", CASES + LARGE)
@pytest.mark.parametrize("pad", [0, 24])
def test_dgrad(sizes, N, K, pad):
    ends, off = _setup(sizes)
    dy, w = _bf16((ends[-1], N), 3), _bf16((len(sizes), N, K), 4)
    ref, mag = _products(ends, dy, w)
    out = torch.full((ends[-1], K + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mx.mx_grouped_gemm_bf16_dgrad(_strided(dy, pad, 8 if pad else 0), w.cuda(), off, dx=out[:, :K])
    _check(got, ref, mag, N, True)
    assert (out[:, K:] == 7.0).all()


@pytest.mark.parametrize("sizes,N,K", CASES + LARGE)
@pytest.mark.parametrize("kind", ["bf16", "fp32", "add"])
@pytest.mark.parametrize("pad", [0, 24])
def test_wgrad(sizes, N, K, kind, pad):
    ends, off = _setup(sizes)
    dy, x = _bf16((ends[-1], N), 5), _bf16((ends[-1], K), 6)
    G = len(sizes)
    old = torch.randn((G, N, K), generator=torch.Generator().manual_seed(7))
    dw = old.cuda() if kind == "add" else torch.full((G, N, K), 7.0, device="cuda",
                                                      dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
    got = mx.mx_grouped_gemm_bf16_wgrad(_strided(dy, pad, 8 if pad else 0), _strided(x, pad), off, dw=dw,
                                        accumulate=kind == "add")
    assert got is dw
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        ref = dy[s:e].double().t() @ x[s:e].double()
        mag = dy[s:e].double().abs().t() @ x[s:e].double().abs()
        if kind == "add":
            ref, mag = ref + old[g].double(), mag + old[g].double().abs()
            if s == e:
                assert torch.equal(got[g].cpu(), old[g])
        _check(got[g], ref, mag, e - s, kind == "bf16")


# long groups and few weights: the rows shared out and joined, with slices that end short or empty
SPLIT = [([3000], 8, 24), ([5000, 0, 1, 3400], 136, 72), ([129, 4000], 264, 200)]


@pytest.mark.parametrize("sizes,N,K", SPLIT)
@pytest.mark.parametrize("kind", ["bf16", "fp32", "add"])
def test_wgrad_shared_out(sizes, N, K, kind):
    ends, off = _setup(sizes)
    G, M = len(sizes), ends[-1]
    need = mx.mx_grouped_gemm_bf16_wgrad_workspace_bytes(G, M, N, K)
    assert need > 0
    test_wgrad(sizes, N, K, kind, 24)
    dy, x = _bf16((M, N), 5).cuda(), _bf16((M, K), 6).cuda()
    outs = []
    for size in (need, need, need - 1):  # a workspace that is too small is not used
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN
        dw = torch.ones((G, N, K), device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
        mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=dw, accumulate=kind == "add", workspace=ws[:size])
        assert (ws[need:] == 255).all()
        assert size == need or (ws == 255).all()
        outs.append(dw)
    assert torch.equal(outs[0], outs[1])
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        ref = dy[s:e].double().cpu().t() @ x[s:e].double().cpu()
        mag = dy[s:e].double().cpu().abs().t() @ x[s:e].double().cpu().abs()
        if kind == "add":
            ref, mag = ref + 1, mag + 1
        _check(outs[2][g], ref, mag, e - s, kind == "bf16")


def test_rows_outside_the_groups_are_left_alone_and_malformed_offsets_stay_in_bounds():
    x, w = _bf16((300, 64), 8).cuda(), _bf16((3, 72, 64), 9).cuda()
    off = torch.tensor([10, 60, 60, 200], dtype=torch.int32, device="cuda")
    out = torch.full((300, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_grouped_gemm_bf16(x, w, off, out=out)
    assert (out[:10] == 7.0).all() and (out[200:] == 7.0).all() and not (out[10:200] == 7.0).all()
    wrong = torch.tensor([-5, 400, 100, 1 << 30], dtype=torch.int32, device="cuda")
    mx.mx_grouped_gemm_bf16(x, w, wrong, out=out)
    mx.mx_grouped_gemm_bf16_dgrad(out, w, wrong)
    mx.mx_grouped_gemm_bf16_wgrad(out, x, wrong)
    torch.cuda.synchronize()


def test_infinite_and_nan_rows_stay_in_their_rows():
    ends, off = _setup([100, 60, 140])
    x, w = _bf16((300, 136), 10), _bf16((3, 72, 136), 11)
    clean = mx.mx_grouped_gemm_bf16(x.cuda(), w.cuda(), off)
    x[101], x[99, 3], x[299, 135] = float("nan"), float("inf"), float("-inf")
    got = mx.mx_grouped_gemm_bf16(x.cuda(), w.cuda(), off)
    keep = torch.ones(300, dtype=torch.bool)
    keep[[99, 101, 299]] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert not got.cpu()[~keep].isfinite().any()


def test_malformed_offsets_with_many_overlapping_groups_end():
    """Offsets that go back and forth make every other group the whole
    matrix: the work is cut off at what valid offsets can give."""
    G, M = 300, 4096
    x, w = _bf16((M, 16), 20).cuda(), _bf16((G, 512, 16), 21).cuda()
    off = torch.tensor([(g % 2) * M for g in range(G + 1)], dtype=torch.int32, device="cuda")
    out = mx.mx_grouped_gemm_bf16(x, w, off)
    mx.mx_grouped_gemm_bf16_dgrad(out, w, off)
    mx.mx_grouped_gemm_bf16_wgrad(out, x, off)
    torch.cuda.synchronize()


def test_operands_past_2_31_elements_and_4_gib():
    """x [300000, 8192] (4.9 GB): rows at both ends and around element 2^31
    and byte 2^32, and the weight gradient of a group past them."""
    M, K, N = 300000, 8192, 16
    ends, off = _setup([100000, 200000 - 37, 37])
    gen = torch.Generator(device="cuda").manual_seed(22)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w, dy = _bf16((3, N, K), 23).cuda(), _bf16((M, N), 24).cuda()
    out = mx.mx_grouped_gemm_bf16(x, w, off)
    dx = mx.mx_grouped_gemm_bf16_dgrad(dy, w, off)
    dw = mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=torch.empty((3, N, K), device="cuda"))
    at = 2 ** 31 // K
    for r in (0, 99990, at - 3, at + 3, M - 45, M - 8):
        rows = slice(r, r + 8)
        g = torch.tensor([sum(e <= i for e in ends[1:]) for i in range(r, r + 8)])
        xr, dyr, wg = x[rows].double().cpu(), dy[rows].double().cpu(), w.double().cpu()[g]
        _check(out[rows], (wg @ xr[:, :, None])[:, :, 0], (wg.abs() @ xr.abs()[:, :, None])[:, :, 0], K, True)
        _check(dx[rows], (dyr[:, None] @ wg)[:, 0], (dyr.abs()[:, None] @ wg.abs())[:, 0], N, True)
    last = slice(ends[2], M)
    a, b = dy[last].double().cpu(), x[last].double().cpu()
    _check(dw[2], a.t() @ b, a.abs().t() @ b.abs(), 37, False)
    cols = slice(8184, 8192)
    a, b = dy[ends[1]:ends[2]].double(), x[ends[1]:ends[2], cols].double()
    _check(dw[1][:, cols], (a.t() @ b).cpu(), (a.abs().t() @ b.abs()).cpu(), ends[2] - ends[1], False)


def test_empty_sizes():
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    w = _bf16((2, 16, 24), 12).cuda()
    assert mx.mx_grouped_gemm_bf16(torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), w, off).shape == (0, 16)
    dw = mx.mx_grouped_gemm_bf16_wgrad(torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"),
                                       torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), off,
                                       dw=torch.ones((2, 16, 24), device="cuda"))
    assert (dw == 0).all()
    # an empty contraction: zeros
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    out = mx.mx_grouped_gemm_bf16(torch.empty((5, 0), dtype=torch.bfloat16, device="cuda"),
                                  torch.empty((2, 16, 0), dtype=torch.bfloat16, device="cuda"), off,
                                  out=torch.ones((5, 16), dtype=torch.bfloat16, device="cuda"))
    assert (out == 0).all()


def test_gradients_against_differences():
    """d sum(out * c) by dgrad and wgrad against central differences of the
    forward's own float64 definition, and of the kernel's forward on exactly
    representable steps."""
    ends, off = _setup([5, 0, 12])
    M, N, K = 17, 16, 24
    # small integers: every product, sum and difference below is exact in fp32 and bf16
    gen = torch.Generator().manual_seed(13)
    x, w, c = (torch.randint(-2, 3, s, generator=gen).float() for s in ((M, K), (3, N, K), (M, N)))

    def loss(x, w):
        out = mx.mx_grouped_gemm_bf16(x.bfloat16().cuda(), w.bfloat16().cuda(), off)
        return float((out.double().cpu() * c.double()).sum())

    dx = mx.mx_grouped_gemm_bf16_dgrad(c.bfloat16().cuda(), w.bfloat16().cuda(), off).float().cpu()
    dw = mx.mx_grouped_gemm_bf16_wgrad(c.bfloat16().cuda(), x.bfloat16().cuda(), off).float().cpu()
    for i, j in ((0, 0), (4, 23), (5, 7), (16, 11)):
        step = torch.zeros_like(x)
        step[i, j] = 1.0
        assert (loss(x + step, w) - loss(x - step, w)) / 2 == dx[i, j]
    for g, i, j in ((0, 0, 0), (0, 15, 23), (1, 3, 3), (2, 7, 9)):
        step = torch.zeros_like(w)
        step[g, i, j] = 1.0
        assert (loss(x, w + step) - loss(x, w - step)) / 2 == dw[g, i, j]


def test_same_bits_every_time_and_on_another_stream():
    ends, off = _setup([300, 0, 513, 87])
    x, w, dy = _bf16((900, 392), 14).cuda(), _bf16((4, 264, 392), 15).cuda(), _bf16((900, 264), 16).cuda()
    first = [mx.mx_grouped_gemm_bf16(x, w, off), mx.mx_grouped_gemm_bf16_dgrad(dy, w, off),
             mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=torch.empty((4, 264, 392), device="cuda"))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [mx.mx_grouped_gemm_bf16(x, w, off, stream=side), mx.mx_grouped_gemm_bf16_dgrad(dy, w, off, stream=side),
             mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=torch.empty((4, 264, 392), device="cuda"), stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_refusals():
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    x, w = _bf16((4, 16), 17).cuda(), _bf16((1, 8, 16), 18).cuda()
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_bf16(x[:, :8], w, off)
    with pytest.raises(TypeError):
        mx.mx_grouped_gemm_bf16(x.float(), w, off)
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_bf16(x, w, off.long())
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_bf16(x, w.cpu(), off)
    with pytest.raises(mx.MxError):
        mx.mx_grouped_gemm_bf16(x[:, :12], _bf16((1, 8, 12), 19).cuda(), off)  # K % 8
    with pytest.raises(mx.MxError):
        mx.mx_grouped_gemm_bf16_wgrad(x, x, off, dw=torch.zeros((1, 16, 16), dtype=torch.bfloat16, device="cuda"),
                                      accumulate=True)
    with pytest.raises(ValueError):
        mx.mx_grouped_gemm_bf16_wgrad(x, x, off, accumulate=True)
