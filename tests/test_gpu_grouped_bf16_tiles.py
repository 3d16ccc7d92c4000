"""Every kernel of the bf16 grouped products with several tiles per workgroup
and full outputs, against float64 products on the GPU.

The launch rules, on 256 CUs: forward and dgrad take 256 x 256 tiles from 192
of them (an upper bound over the rows' distribution) and more than 128 rows a
group on average, else 128 x 128 ones with two stages in LDS (more than 256
tiles) or four; the weight gradient from 192 and 1024 rows a group, or from
1024 tiles.  A launch of large tiles has at most 256 workgroups, of small ones
512.  Tolerances: tests/test_gpu_grouped_bf16.py."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from test_gpu_grouped_bf16 import _check, _setup

pytestmark = pytest.mark.gpu


def _bf16(shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def _tiles(n, t):
    return -(-n // t)


def _row_tiles(sizes, t):
    return sum(_tiles(s, t) for s in sizes)


def _skewed(G, M, seed):
    """G group sizes with a long tail and empty ones, M in all."""
    r = np.random.Generator(np.random.PCG64(seed))
    p = (1.0 + np.arange(G)) ** -1.1
    p[r.permutation(G)[:G // 8]] = 0
    return r.multinomial(M, r.permutation(p / p.sum())).tolist()


def _grouped(ends, a, b):
    """Rows of a group times b[g], and the same of magnitudes: float64, on the GPU."""
    width = b.shape[2]
    ref, mag = (torch.empty((a.shape[0], width), dtype=torch.float64, device="cuda") for _ in range(2))
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        if e > s:
            x, w = a[s:e].double(), b[g].double()
            ref[s:e] = x @ w
            mag[s:e] = x.abs() @ w.abs()
    return ref, mag


# group sizes around a tile's (row ends at 1, 127, 128, 129, 255 and 256 past a tile among them)
EDGES = [1500, 0, 33, 2600, 900, 1, 511, 2047, 257, 383, 384, 385, 767, 768]
# (sizes, N, K, tile): large tiles in several rounds; small tiles, two stages, several rounds; small tiles, four stages
FORWARD = [
    (EDGES, 2568, 328, 256),
    ([70, 128, 0, 127, 1, 250, 129] * 8, 1544, 200, 128),
    ([130, 0, 96, 256, 3], 1032, 392, 128),
    (_skewed(300, 9000, 1), 392, 136, 128),    # more groups than threads of a workgroup
    (_skewed(600, 12000, 2), 264, 72, 128),
    (_skewed(4096, 65536, 3), 24, 40, 128),    # as many groups as are accepted
    ([600] * 300, 136, 72, 256),               # large tiles, more groups than threads
]


@pytest.mark.parametrize("k", range(len(FORWARD)))
@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_forward_and_dgrad(direction, k):
    sizes, N, K, tile = FORWARD[k]
    ends, off = _setup(sizes)
    G, M = len(sizes), ends[-1]
    width, depth = (N, K) if direction == "forward" else (K, N)
    if direction == "dgrad":  # the same output widths
        N, K, width, depth = K, N, N, K
    # the kernel that the sizes are meant for
    bound = (_tiles(M, 256) + min(G, M)) * _tiles(width, 256)
    assert (bound >= 192 and M > 128 * G) == (tile == 256) and not (M <= 8 * G or M <= 64)
    actual = _row_tiles(sizes, tile) * _tiles(width, tile)
    if k in (0, 1, 6):
        assert actual > 1.5 * (256 if tile == 256 else 512)
    w = _bf16((G, N, K), 2)
    out = torch.full((M, width), 7.0, dtype=torch.bfloat16, device="cuda")
    if direction == "forward":
        a = _bf16((M, K), 1)
        mx.mx_grouped_gemm_bf16(a, w, off, out=out)
        ref, mag = _grouped(ends, a, w.transpose(1, 2))
    else:
        a = _bf16((M, N), 1)
        mx.mx_grouped_gemm_bf16_dgrad(a, w, off, dx=out)
        ref, mag = _grouped(ends, a, w)
    _check(out, ref.cpu(), mag.cpu(), depth, True)


# few rows a group on average, with uneven groups and more of them than threads of a workgroup (512)
FEW = [(_skewed(600, 4000, 4), 136, 264), (_skewed(4096, 20000, 5), 24, 72), ([1000] + [0] * 127, 520, 1032),
       ([0] * 4095 + [64], 40, 136)]


@pytest.mark.parametrize("sizes,N,K", FEW)
def test_few_rows_with_many_groups(sizes, N, K):
    ends, off = _setup(sizes)
    G, M = len(sizes), ends[-1]
    assert M <= 8 * G
    x, w = _bf16((M, K), 3), _bf16((G, N, K), 4)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_grouped_gemm_bf16(x, w, off, out=out)
    ref, mag = _grouped(ends, x, w.transpose(1, 2))
    _check(out, ref.cpu(), mag.cpu(), K, True)


WGRAD = [
    ([3000, 0, 1, 1500, 700], 2056, 2312, 256),      # large tiles, several rounds, skewed and empty groups
    ([70, 1027, 0, 513, 64, 65, 1, 3], 2056, 1544, 128),  # small tiles, two stages, several rounds
    ([130, 0, 96, 256, 3], 392, 520, 128),           # small tiles, four stages
    (_skewed(300, 4000, 6), 264, 136, 128),          # more groups than threads of a workgroup
    (_skewed(600, 5000, 7), 136, 72, 128),           # more than are taken longest first
    (_skewed(1100, 9000, 8), 24, 40, 256),           # the same, large tiles
    (_skewed(4096, 20000, 9), 16, 24, 256),          # as many groups as are accepted
]


@pytest.mark.parametrize("k", range(len(WGRAD)))
@pytest.mark.parametrize("kind", ["bf16", "fp32", "add"])
def test_wgrad(kind, k):
    sizes, N, K, tile = WGRAD[k]
    ends, off = _setup(sizes)
    G, M = len(sizes), ends[-1]
    tiles = G * _tiles(N, 256) * _tiles(K, 256)
    assert (tiles >= 192 and (tiles >= 1024 or M >= 1024 * G)) == (tile == 256)
    assert mx.mx_grouped_gemm_bf16_wgrad_workspace_bytes(G, M, N, K) == 0  # not shared out
    if k in (0, 1):
        assert G * _tiles(N, tile) * _tiles(K, tile) > 1.5 * (256 if tile == 256 else 512)
    dy, x = _bf16((M, N), 5), _bf16((M, K), 6)
    old = torch.randn((G, N, K), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    dw = old.clone() if kind == "add" else torch.full((G, N, K), 7.0, device="cuda",
                                                       dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
    mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=dw, accumulate=kind == "add")
    ref, mag = (torch.zeros((G, N, K), dtype=torch.float64, device="cuda") for _ in range(2))
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        if e > s:
            a, b = dy[s:e].double().t().contiguous(), x[s:e].double()
            ref[g], mag[g] = a @ b, a.abs() @ b.abs()
    if kind == "add":
        ref, mag = ref + old.double(), mag + old.double().abs()
        empty = [g for g, n in enumerate(sizes) if n == 0]
        assert torch.equal(dw[empty], old[empty])
    for part in ([slice(g, g + 1) for g in range(G)] if G < 16 else [slice(0, G)]):
        longest = max(sizes[part])
        _check(dw[part], ref[part].cpu(), mag[part].cpu(), longest, kind == "bf16")


# rows shared out: (group sizes, N, K, slices, tile)
SHARED = [([90000, 0, 1, 60000, 33000, 70000, 20, 16979], 128, 120, 32, 256), ([50000, 0, 1, 3400], 136, 72, 13, 128),
          ([30000, 1, 0, 2769], 512, 512, 8, 128)]


@pytest.mark.parametrize("sizes,N,K,slices,tile", SHARED)
@pytest.mark.parametrize("kind", ["bf16", "fp32", "add"])
def test_wgrad_with_rows_shared_out(sizes, N, K, slices, tile, kind):
    ends, off = _setup(sizes)
    G, M = len(sizes), ends[-1]
    need = mx.mx_grouped_gemm_bf16_wgrad_workspace_bytes(G, M, N, K)
    assert need == 4 * slices * G * N * K
    tiles = slices * G * _tiles(N, 256) * _tiles(K, 256)  # the kernel that the slices are meant for
    assert (tiles >= 192 and (tiles >= 1024 or M >= 1024 * slices * G)) == (tile == 256)
    dy, x = _bf16((M, N), 11), _bf16((M, K), 12)
    old = torch.randn((G, N, K), generator=torch.Generator(device="cuda").manual_seed(13), device="cuda")
    dw = old.clone() if kind == "add" else torch.full((G, N, K), 7.0, device="cuda",
                                                       dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
    mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=dw, accumulate=kind == "add")
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        a, b = dy[s:e].double().t().contiguous(), x[s:e].double()
        ref, mag = a @ b, a.abs() @ b.abs()
        if kind == "add":
            ref, mag = ref + old[g].double(), mag + old[g].double().abs()
        _check(dw[g], ref.cpu(), mag.cpu(), e - s + slices, kind == "bf16")


@pytest.mark.parametrize("rows", [6, 1200])
def test_weights_past_2_31_elements_and_4_gib(rows):
    """w and dw [33, 8192, 8192] (2.2 10^9 elements): the last group's
    products, by few rows and by tiles, and the first group's."""
    G, N, K = 33, 8192, 8192
    sizes = [0] * G
    sizes[0], sizes[G - 2], sizes[G - 1] = rows // 2, 1, rows // 3
    ends, off = _setup(sizes)
    M = ends[-1]
    gen = torch.Generator(device="cuda").manual_seed(8)
    w = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda")
    for g in range(G):
        w[g].normal_(generator=gen)
    x, dy = _bf16((M, K), 9), _bf16((M, N), 10)
    out, dx = mx.mx_grouped_gemm_bf16(x, w, off), mx.mx_grouped_gemm_bf16_dgrad(dy, w, off)
    for g in (0, G - 2, G - 1):
        s, e = ends[g], ends[g + 1]
        wg = w[g].double()
        a, b = x[s:e].double(), dy[s:e].double()
        _check(out[s:e], (a @ wg.t()).cpu(), (a.abs() @ wg.abs().t()).cpu(), K, True)
        _check(dx[s:e], (b @ wg).cpu(), (b.abs() @ wg.abs()).cpu(), N, True)
    del w
    dw = torch.full((G, N, K), 7.0, device="cuda")
    mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, dw=dw)
    assert (dw[1:G - 2] == 0).all()
    for g in (0, G - 2, G - 1):
        a, b = dy[ends[g]:ends[g + 1]].double().t().contiguous(), x[ends[g]:ends[g + 1]].double()
        ref, mag = a @ b, a.abs() @ b.abs()
        e = (sizes[g] + 1) * 2.0 ** -23 * mag
        assert not ((dw[g].double() - ref).abs() > e + 2.0 ** -23 * ref.abs()).any()
