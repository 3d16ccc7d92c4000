"""The norm and its gradients on batches: several rounds of the persistent
loop for every width of a row's team, calls whose rows pass the caches, and
sums of many waves."""
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from test_gpu_rms_norm import EPS, TYPES, U, _check_gradients, _check_y

pytestmark = pytest.mark.gpu


def _randn(gen, M, N, kind="bf16", scale=1.0):
    return (torch.randn((M, N), generator=gen, device="cuda") * scale).to(TYPES[kind])


@pytest.mark.parametrize("N,small", [(16384, 1.375 * 2.0 ** -13), (32768, 0.96875 * 2.0 ** -13)])
def test_small_waves_beside_a_large_one(N, small):
    """One wave's part of the sum is 512, the 15 others' 0.94 of half a step of it each."""
    x = torch.full((3, N), small, dtype=torch.bfloat16, device="cuda")
    x[:, :512] = 1.0
    rstd = mx.mx_rms_norm(x, torch.ones(N, device="cuda"), eps=0.0, y=None, rstd=True)[4]
    want = 1 / x.double().square().mean(1).sqrt()
    # joined in pairs at most two such parts meet the large one alone, and 3 roundings are below half a step: 3 half steps
    # of the sum, half of that in r; the mean is exact, the square root and the quotient are half a step off each
    assert ((rstd.double() - want).abs() <= want * U * (1.5 + 2)).all()


def _forward(gen, M, N, stream, weight, quant):
    x = _randn(gen, M, N)
    residual = None if stream == "none" else _randn(gen, M, N, stream, 3.0)
    w = (1 + 0.3 * torch.randn(N, generator=gen, device="cuda")).to(TYPES[weight])
    y, h, q, s, rstd = mx.mx_rms_norm(x, w, residual=residual, eps=EPS, q=True if quant else None, rstd=True)
    if residual is None:
        h = x
    else:
        assert torch.equal(h, (x.float() + residual.float()).to(residual.dtype))
    for at in range(0, M, max(1, (1 << 24) // N)):  # (a part at a time: float64)
        rows = slice(at, at + max(1, (1 << 24) // N))
        _check_y(y[rows], rstd[rows], h[rows], w)
    if quant:
        qy, sy = mx.mx_quantize_rows(y)
        assert torch.equal(q, qy) and torch.equal(s, sy)


@pytest.mark.parametrize("M,N,stream,quant", [
    (4701, 7168, "bf16", True), (4701, 7168, "fp32", True), (4690, 7168, "none", True), (8209, 4096, "bf16", True),
    (2051, 16384, "bf16", True), (1037, 32768, "bf16", True), (17001, 2080, "fp32", True), (32801, 1056, "bf16", True),
    (33001, 1024, "bf16", True), (66001, 512, "none", True), (131301, 256, "bf16", True), (262501, 128, "fp32", True),
    (525001, 64, "bf16", True), (24001, 1400, "bf16", False)])
def test_rows_that_pass_the_caches(M, N, stream, quant):
    gen = torch.Generator(device="cuda").manual_seed(M)
    _forward(gen, M, N, stream, "bf16" if M % 2 else "fp32", quant)


@pytest.mark.parametrize("M,N", [
    (20001, 64), (9001, 128), (5001, 256), (3001, 512), (3001, 1000),  # several teams a workgroup, two rounds and more
    (8193, 1480), (3001, 1480), (1700, 2056), (1300, 4104), (700, 9000), (600, 20000),  # a workgroup a row
    (4701, 7168), (16601, 2048), (2051, 16384), (1031, 32768), (525001, 64), (66001, 512), (23001, 1480)])  # past the caches
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradients_of_batches(kind, M, N):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    h, dy = _randn(gen, M, N, kind, 2.0), _randn(gen, M, N)
    dy2, dh_in = _randn(gen, M, N, scale=0.3), _randn(gen, M, N, kind)
    weight = (1 + 0.3 * torch.randn(N, generator=gen, device="cuda")).to(TYPES["bf16" if M % 4 == 1 else "fp32"])
    rstd = mx.mx_rms_norm(h, weight, eps=EPS, y=None, rstd=True)[4]
    for second, stream in ((dy2, dh_in), (None, None)):
        dh, dx, dw = mx.mx_rms_norm_backward(dy, h, weight, rstd, dy2=second, dh_in=stream, dweight=torch.float32,
                                             dx=True if kind == "fp32" else None)
        step = max(1, (1 << 24) // N)
        want, mag = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
        for at in range(0, M, step):
            rows = slice(at, at + step)
            part = [None if t is None else t[rows] for t in (dy, h, rstd, second, stream, dh, dx)]
            _check_gradients((part[5], part[6], None), part[0], part[1], weight, part[2], part[3], part[4])
            g = part[0].double() + (0 if second is None else part[3].double())
            z = part[1].double() * part[2].double()[:, None]
            want += (g * z).sum(0)
            mag += (g * z).abs().sum(0)
        # a team adds M / 256 rows in a row at most, up to 1024 parts and 32 teams of each are added after; 6 roundings
        # besides
        rel = U * (min(M, M / 256 + 1024 + 32) + 6)
        assert ((dw.double() - want).abs() <= mag * rel + 2.0 ** -133).all()


def test_replacing_inputs_past_the_caches():
    gen = torch.Generator(device="cuda").manual_seed(3)
    M, N = 4701, 7168
    t = {n: _randn(gen, M, N) for n in ("h", "dy", "dy2", "dh_in")}
    weight = torch.randn(N, generator=gen, device="cuda")
    rstd = mx.mx_rms_norm(t["h"], weight, eps=EPS, y=None, rstd=True)[4]
    want = mx.mx_rms_norm_backward(t["dy"], t["h"], weight, rstd, dy2=t["dy2"], dh_in=t["dh_in"], dweight=torch.float32)
    for what in t:
        fresh = {n: v.clone() for n, v in t.items()}
        got = mx.mx_rms_norm_backward(fresh["dy"], fresh["h"], weight, rstd, dy2=fresh["dy2"], dh_in=fresh["dh_in"],
                                      dh=fresh[what], dweight=torch.float32)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    x, residual = t["dy"], t["dh_in"]
    y, h, _, _, r = mx.mx_rms_norm(x, weight, residual=residual, eps=EPS, rstd=True)
    into = x.clone()
    got = mx.mx_rms_norm(into, weight, residual=residual, h=residual, y=into, eps=EPS, rstd=True)
    assert torch.equal(into, y) and torch.equal(residual, h) and torch.equal(got[4], r)
