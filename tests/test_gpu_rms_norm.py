"""The root-mean-square norm, its MXFP8 rows and its gradients against the
formulas in float64, at the sizes, types and strides where they can go wrong."""
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of float32, relative
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6

WIDTHS = [8, 32, 96, 128, 136, 160, 256, 264, 288, 512, 520, 1000, 1024, 1032, 1056, 2048, 2080, 4096, 7168, 8192,
          8200, 8224, 12320, 16384, 16392, 16416, 32768]


def _rows(gen, M, N, kind, ld=None, scale=1.0):
    whole = torch.full((M, ld or N), float("nan"), dtype=TYPES[kind], device="cuda")
    whole[:, :N] = (torch.randn((M, N), generator=gen) * scale).to(TYPES[kind]).cuda()
    return whole[:, :N]


def _half_step(t):
    return torch.finfo(t.dtype).eps / 2


def _check_y(y, rstd, h, weight):
    v, w = h.double(), weight.double()
    r = 1 / (v.square().mean(1) + EPS).sqrt()
    N = h.shape[1]
    # a lane squares and adds N / 16 values in a row at most, 12 joins; half of it reaches r, with 4 roundings of r and 2
    # of the products
    rel = U * (8 + N / 32 + 12)
    if rstd is not None:
        assert ((rstd.double() - r).abs() <= r * rel).all()
    if y is not None:
        want = v * r[:, None] * w
        assert ((y.double() - want).abs() <= want.abs() * (_half_step(y) + rel) + 2.0 ** -133).all()


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("stream", ["none", "bf16", "fp32"])
def test_norm(stream, N):
    M = 37 if N <= 8192 else 5
    gen = torch.Generator().manual_seed(N)
    x = _rows(gen, M, N, "bf16")
    residual = None if stream == "none" else _rows(gen, M, N, stream, scale=3.0)
    weight = (1 + 0.3 * torch.randn(N, generator=gen)).to(TYPES["fp32" if N % 64 else "bf16"]).cuda()
    quant = N % 32 == 0
    y, h, q, s, rstd = mx.mx_rms_norm(x, weight, residual=residual, eps=EPS, q=True if quant else None, rstd=True)
    if residual is None:
        assert h is None
        h = x
    else:
        assert torch.equal(h, (x.float() + residual.float()).to(residual.dtype))
    _check_y(y, rstd, h, weight)
    if quant:
        qy, sy = mx.mx_quantize_rows(y)
        assert torch.equal(q, qy) and torch.equal(s, sy)
    # the outputs do not depend on what else is written
    alone = mx.mx_rms_norm(x, weight, residual=residual, eps=EPS, y=None, q=True if quant else None)
    assert alone[0] is None and alone[4] is None
    if residual is not None:
        assert torch.equal(alone[1], h)
    if quant:
        assert torch.equal(alone[2], q) and torch.equal(alone[3], s)
    # the norm of the sum is the norm of the stream
    again = mx.mx_rms_norm(h, weight, eps=EPS, rstd=True)
    assert torch.equal(again[0], y) and torch.equal(again[4], rstd)


@pytest.mark.parametrize("M", [1, 2, 31, 32, 33, 64, 100, 1025])
@pytest.mark.parametrize("N", [32, 128, 224, 512, 1024, 2304])
def test_every_number_of_rows_and_the_scales_padding(N, M):
    gen = torch.Generator().manual_seed(M)
    x, weight = _rows(gen, M, N, "bf16"), torch.randn(N, generator=gen).cuda()
    size = mx.mx_scale_bytes(M, N)
    s = torch.full((size + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    q = torch.full((M + 2, N), 0xEE, dtype=torch.uint8, device="cuda")
    rstd = torch.full((M + 2,), 7.0, device="cuda")
    y = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_rms_norm(x, weight, eps=EPS, y=y[:M], q=q[:M], s=s[:size], rstd=rstd[:M])
    _check_y(y[:M], rstd[:M], x, weight)
    qy, sy = mx.mx_quantize_rows(y[:M])
    assert torch.equal(q[:M], qy) and torch.equal(s[:size], sy)
    assert (s[size:] == 0xEE).all() and (q[M:] == 0xEE).all() and (rstd[M:] == 7).all() and (y[M:] == 7).all()


@pytest.mark.parametrize("N", [64, 520, 2048, 16392])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_strides_and_in_place(kind, N):
    gen = torch.Generator().manual_seed(5)
    x, residual = _rows(gen, 21, N, "bf16", N + 8), _rows(gen, 21, N, kind, N + 16)
    weight = torch.randn(N, generator=gen).cuda()
    want = mx.mx_rms_norm(x.contiguous(), weight, residual=residual.contiguous())
    out = torch.full((21, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((21, N + 32), 7.0, dtype=TYPES[kind], device="cuda")
    mx.mx_rms_norm(x, weight, residual=residual, h=h[:, :N], y=out[:, :N])
    assert torch.equal(out[:, :N], want[0]) and torch.equal(h[:, :N], want[1])
    assert (out[:, N:] == 7).all() and (h[:, N:] == 7).all()
    mx.mx_rms_norm(x, weight, residual=residual, h=residual, y=x)
    assert torch.equal(x, want[0]) and torch.equal(residual, want[1])


@pytest.mark.parametrize("N", [64, 1024, 7168])
def test_zeros_large_and_small_values(N):
    x = torch.zeros((6, N), dtype=torch.bfloat16, device="cuda")
    x[1, 3] = 2.0 ** 60     # one value has it all
    x[2] = 2.0 ** -60       # far below eps
    x[3] = 2.0 ** 50
    x[4, ::2], x[4, 1::2] = 2.0 ** 20, -(2.0 ** -20)
    weight = torch.ones(N, device="cuda")
    y, _, _, _, rstd = mx.mx_rms_norm(x, weight, eps=EPS, rstd=True)
    _check_y(y, rstd, x, weight)
    assert (y[0] == 0).all() and (y[5] == 0).all()


def test_not_finite_rows_stay_in_their_rows():
    gen = torch.Generator().manual_seed(6)
    x, weight = _rows(gen, 9, 512, "bf16"), torch.ones(512, device="cuda")
    clean = mx.mx_rms_norm(x, weight)[0]
    x[2, 7], x[5, 100] = float("nan"), float("inf")
    y = mx.mx_rms_norm(x, weight)[0]
    for r in range(9):
        if r == 2:
            assert y[r].isnan().all()
        elif r == 5:
            assert (y[r, :100] == 0).all() and y[r, 100].isnan()
        else:
            assert torch.equal(y[r], clean[r])


def test_rows_past_2_31_elements():
    ld, M, N = 1 << 26, 40, 264
    wide = [torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").as_strided((M, N), (ld, 1)) for _ in range(2)]
    gen = torch.Generator().manual_seed(7)
    x, weight = _rows(gen, M, N, "bf16"), torch.randn(N, generator=gen).cuda()
    for w in wide:
        w.copy_(x)
    want = mx.mx_rms_norm(x, weight, residual=x, rstd=True)
    y, h, _, _, rstd = mx.mx_rms_norm(wide[0], weight, residual=wide[1], h=wide[1], y=wide[0], rstd=True)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    dy = _rows(gen, M, N, "bf16")
    grads = mx.mx_rms_norm_backward(dy, want[1], weight, rstd, dh_in=dy)
    wide[0].copy_(dy)
    got = mx.mx_rms_norm_backward(wide[0], h, weight, rstd, dh_in=wide[0], dh=wide[0])
    assert torch.equal(got[0], grads[0]) and torch.equal(got[2], grads[2])


def test_many_short_rows():
    """More rows than workgroups in one round of the grid."""
    M, N = (1 << 24) + 333, 16
    x = torch.randn((M, N), device="cuda", dtype=torch.bfloat16)
    weight = torch.randn(N, device="cuda")
    y, _, _, _, rstd = mx.mx_rms_norm(x, weight, eps=EPS, rstd=True)
    for part in (slice(0, 70000), slice(M - 70000, M)):
        _check_y(y[part], rstd[part], x[part], weight)
    assert mx.mx_rms_norm(x[:0], weight)[0].shape == (0, N)


# -- gradients ------------------------------------------------------------------


def _check_gradients(got, dy, h, weight, rstd, dy2, dh_in, before=None, split=512):
    dh, dx, dw = got
    g = dy.double() + (0 if dy2 is None else dy2.double())
    r = rstd.double()[:, None]
    M, N = h.shape
    z, a = h.double() * r, g * weight.double()
    mean = (a * z).mean(1, keepdim=True)
    want = r * (a - z * mean)
    mag = r * (a.abs() + z.abs() * (a * z).abs().mean(1, keepdim=True))
    if dh_in is not None:
        want, mag = want + dh_in.double(), mag + dh_in.double().abs()
    # fp32: a lane adds N / 16 products in a row at most, 12 joins, 8 roundings besides (g's among them)
    rel = U * (8 + N / 16 + 12)
    assert ((dh.double() - want).abs() <= mag * rel + want.abs() * _half_step(dh) + 2.0 ** -133).all()
    if dx is not None:
        assert torch.equal(dx, dh.to(torch.bfloat16))
    if dw is not None:
        terms = g * z
        want, mag = terms.sum(0), terms.abs().sum(0)
        if before is not None:
            want, mag = want + before.double(), mag + before.double().abs()
        # a part adds M / parts rows in a row, then the parts are added: M at most, for few rows; 6 roundings besides
        rel = U * (min(M, M / split + split) + 6)
        assert ((dw.double() - want).abs() <= mag * rel + want.abs() * _half_step(dw) + 2.0 ** -133).all()


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradients(kind, N):
    M = 37 if N <= 8192 else 5
    gen = torch.Generator().manual_seed(N + 1)
    h, dy, dy2 = _rows(gen, M, N, kind, scale=2.0), _rows(gen, M, N, "bf16"), _rows(gen, M, N, "bf16", scale=0.3)
    dh_in = _rows(gen, M, N, kind)
    weight = (1 + 0.3 * torch.randn(N, generator=gen)).to(TYPES["bf16" if N % 64 else "fp32"]).cuda()
    rstd = mx.mx_rms_norm(h, weight, eps=EPS, y=None, rstd=True)[4]
    for second, stream in ((None, None), (dy2, dh_in), (None, dh_in), (dy2, None)):
        got = mx.mx_rms_norm_backward(dy, h, weight, rstd, dy2=second, dh_in=stream, dx=True if kind == "fp32" else None)
        assert got[2].dtype == weight.dtype
        _check_gradients(got, dy, h, weight, rstd, second, stream)
    alone = mx.mx_rms_norm_backward(dy, h, weight, rstd, dweight=None)
    assert alone[2] is None and torch.equal(alone[0], mx.mx_rms_norm_backward(dy, h, weight, rstd)[0])


@pytest.mark.parametrize("M", [0, 1, 2, 3, 31, 511, 256, 257, 513, 1025, 5000])
@pytest.mark.parametrize("N", [24, 64, 520, 2056])
def test_weight_gradient_of_every_number_of_rows(N, M):
    gen = torch.Generator().manual_seed(M)
    h, dy = _rows(gen, M, N, "bf16"), _rows(gen, M, N, "bf16")
    weight = torch.randn(N, generator=gen).cuda()
    rstd = mx.mx_rms_norm(h, weight, eps=EPS, y=None, rstd=True)[4]
    for kind in (torch.float32, torch.bfloat16):
        got = mx.mx_rms_norm_backward(dy, h, weight, rstd, dweight=kind)
        assert got[2].dtype == kind
        _check_gradients(got, dy, h, weight, rstd, None, None)
        if M == 0:
            assert (got[2] == 0).all()
    before = torch.randn(N, generator=gen).cuda()
    total = before.clone()
    got = mx.mx_rms_norm_backward(dy, h, weight, rstd, dweight=total, accumulate=True)
    assert got[2] is total
    _check_gradients(got, dy, h, weight, rstd, None, None, before=before)
    if M == 0:
        assert torch.equal(total, before)


@pytest.mark.parametrize("N", [64, 520, 2048, 16392])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradient_strides_and_in_place(kind, N):
    gen = torch.Generator().manual_seed(15)
    h, dy, dy2 = _rows(gen, 21, N, kind, N + 8), _rows(gen, 21, N, "bf16", N + 16), _rows(gen, 21, N, "bf16", N + 24)
    dh_in = _rows(gen, 21, N, kind, N + 40)
    weight = torch.randn(N, generator=gen).cuda()
    rstd = mx.mx_rms_norm(h, weight, y=None, rstd=True)[4]
    want = mx.mx_rms_norm_backward(dy.contiguous(), h.contiguous(), weight, rstd, dy2=dy2.contiguous(),
                                   dh_in=dh_in.contiguous())
    out = torch.full((22, N + 24), 7.0, dtype=TYPES[kind], device="cuda")
    got = mx.mx_rms_norm_backward(dy, h, weight, rstd, dy2=dy2, dh_in=dh_in, dh=out[:21, :N])
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert (out[:, N:] == 7).all() and (out[21] == 7).all()
    if kind == "bf16":
        into = _rows(gen, 21, N, "bf16", N + 16)
        into.copy_(dy)
        mx.mx_rms_norm_backward(into, h, weight, rstd, dy2=dy2, dh_in=dh_in, dh=into)
        assert torch.equal(into, want[0])
    got = mx.mx_rms_norm_backward(dy, h, weight, rstd, dy2=dy2, dh_in=dh_in, dh=dh_in)
    assert torch.equal(dh_in, want[0])


@pytest.mark.parametrize("M", [200, 256, 3000])
@pytest.mark.parametrize("N", [128, 1480, 7168, 16392])
@pytest.mark.parametrize("what", ["dy", "dy2", "h", "dh_in"])
def test_gradients_that_replace_an_input(what, N, M):
    """dweight is that of the inputs that were there, and the others stay."""
    M = M if N <= 7168 else min(M, 300)
    gen = torch.Generator().manual_seed(16)
    t = {n: _rows(gen, M, N, "bf16") for n in ("h", "dy", "dy2", "dh_in")}
    weight = torch.randn(N, generator=gen).cuda()
    rstd = mx.mx_rms_norm(t["h"], weight, eps=EPS, y=None, rstd=True)[4]
    before = {n: v.clone() for n, v in t.items()}
    want = mx.mx_rms_norm_backward(t["dy"], t["h"], weight, rstd, dy2=t["dy2"], dh_in=t["dh_in"], dweight=torch.float32)
    _check_gradients(want, t["dy"], t["h"], weight, rstd, t["dy2"], t["dh_in"])
    got = mx.mx_rms_norm_backward(t["dy"], t["h"], weight, rstd, dy2=t["dy2"], dh_in=t["dh_in"], dh=t[what],
                                  dweight=torch.float32)
    assert torch.equal(t[what], want[0])
    assert all(torch.equal(t[n], before[n]) for n in t if n != what)
    # the same sum, perhaps in the order of another kernel's workgroups: each within its bound of the true one
    _check_gradients((want[0], None, got[2]), before["dy"], before["h"], weight, rstd, before["dy2"], before["dh_in"])


@pytest.mark.parametrize("M", [200, 3000])
@pytest.mark.parametrize("what", ["dy", "dy2"])
def test_the_bf16_gradient_of_a_float32_stream_in_place(what, M):
    gen = torch.Generator().manual_seed(17)
    h, dh_in = _rows(gen, M, 520, "fp32"), _rows(gen, M, 520, "fp32")
    t = {n: _rows(gen, M, 520, "bf16") for n in ("dy", "dy2")}
    weight = torch.randn(520, generator=gen).cuda()
    rstd = mx.mx_rms_norm(h, weight, eps=EPS, y=None, rstd=True)[4]
    before = {n: v.clone() for n, v in t.items()}
    want = mx.mx_rms_norm_backward(t["dy"], h, weight, rstd, dy2=t["dy2"], dh_in=dh_in, dx=True)
    got = mx.mx_rms_norm_backward(t["dy"], h, weight, rstd, dy2=t["dy2"], dh_in=dh_in, dh=dh_in.clone(), dx=t[what])
    assert torch.equal(got[0], want[0]) and torch.equal(t[what], want[1])
    _check_gradients((want[0], None, got[2]), before["dy"], h, weight, rstd, before["dy2"], dh_in)


@pytest.mark.parametrize("N", [16, 640])
def test_gradients_against_differences(N):
    """d/dh and d/dw of sum(dy y) by central differences of the float64 norm of a float32 stream."""
    gen = torch.Generator().manual_seed(25)
    M = 3
    h, dy = _rows(gen, M, N, "fp32"), _rows(gen, M, N, "bf16")
    weight = (1 + 0.3 * torch.randn(N, generator=gen)).cuda()
    rstd = mx.mx_rms_norm(h, weight, eps=EPS, y=None, rstd=True)[4]
    dh, _, dw = mx.mx_rms_norm_backward(dy, h, weight, rstd)

    def value(h, w):
        return (dy.double() * h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * w).sum(1)

    step = 1e-5
    for c in (0, N // 2, N - 1):
        e = torch.zeros(N, dtype=torch.float64, device="cuda")
        e[c] = step
        d = (value(h.double() + e, weight.double()) - value(h.double() - e, weight.double())) / (2 * step)
        assert torch.allclose(dh[:, c].double(), d, rtol=1e-5, atol=1e-5)
        d = (value(h.double(), weight.double() + e) - value(h.double(), weight.double() - e)).sum() / (2 * step)
        assert abs(float(dw[c]) - float(d)) <= 1e-5 * (1 + abs(float(d)))


# -- streams and graphs -----------------------------------------------------------


def test_captured_and_replayed():
    gen = torch.Generator().manual_seed(35)
    M, N = 300, 1056
    x, residual, dy = (_rows(gen, M, N, "bf16") for _ in range(3))
    weight = torch.randn(N, generator=gen).cuda()
    size = mx.mx_rms_norm_backward_workspace_bytes(M, N)

    def make():
        return {"h": torch.zeros_like(x), "y": torch.zeros_like(x), "rstd": torch.zeros(M, device="cuda"),
                "q": torch.zeros((M, N), dtype=torch.uint8, device="cuda"),
                "s": torch.zeros(mx.mx_scale_bytes(M, N), dtype=torch.uint8, device="cuda"),
                "dh": torch.zeros_like(x), "dw": torch.zeros(N, device="cuda"),
                "space": torch.zeros(size, dtype=torch.uint8, device="cuda")}

    def step(o):
        mx.mx_rms_norm(x, weight, residual=residual, h=o["h"], y=o["y"], q=o["q"], s=o["s"], rstd=o["rstd"])
        mx.mx_rms_norm_backward(dy, o["h"], weight, o["rstd"], dh_in=dy, dh=o["dh"], dweight=o["dw"], accumulate=True,
                                workspace=o["space"])

    step(make())
    torch.cuda.synchronize()
    eager, captured = make(), make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for _ in range(4):
        x.copy_(_rows(gen, M, N, "bf16"))
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[n], captured[n]) for n in eager)


def test_on_another_stream_and_the_same_bits():
    gen = torch.Generator().manual_seed(45)
    x, dy = _rows(gen, 3000, 2048, "bf16"), _rows(gen, 3000, 2048, "bf16")
    weight = torch.randn(2048, generator=gen).cuda()
    want = mx.mx_rms_norm(x, weight, residual=dy, q=True, rstd=True)
    grads = mx.mx_rms_norm_backward(dy, want[1], weight, want[4])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        got = mx.mx_rms_norm(x, weight, residual=dy, q=True, rstd=True, stream=stream)
        back = mx.mx_rms_norm_backward(dy, got[1], weight, got[4], stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(back[0], grads[0]) and torch.equal(back[2], grads[2])
