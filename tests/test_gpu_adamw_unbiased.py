"""8-bit AdamW states rounded without bias: right on average where rounding
to nearest holds them, and one step against the formulas.

Tolerances of the averages.  Neighbouring codes are at most 1/8 apart (2^-3
relative), so their squares at most 0.27 v.  Rounding z in [a, b] at random
without bias has the variance (z - a)(b - z).  A step moves a state on a code
c by (1 - b2) |g^2 - c^2|, so it adds at most (1 - b2) |g^2 - c^2| 0.27 c^2;
summed over the steps that a state remembers (1 / (1 - b2^2)) at most
0.138 E(|g^2 - c^2| c^2) for b2 >= 0.95.  With c^2 = v (1 + e), std(e) = s:
constant gradients (g^2 = v): s^2 <= 0.138 s sqrt(1 + s^2), s <= 0.14;
Gaussian ones: s^2 <= 0.138 (2.05 + s^2), s <= 0.57.
m: rounding adds at most (1/16 m)^2 a step, summed 1 / (1 - 0.81): s <= 0.15
of its root mean square.  The elements' roundings are independent: the mean
over N = 64 * 255 = 16320 of them is within 6 s / sqrt(N) except with
probability 10^-8."""
import math

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from mxfp8_block_scaled_04_amd.optimizer import AdamW
from test_gpu_adamw import BLOCK, TINY, U, Tensors, _check, _steps

pytestmark = pytest.mark.gpu

N_BLOCKS = 64
N = N_BLOCKS * BLOCK
SIGMA6 = 6 / math.sqrt(N_BLOCKS * 255)


def _optimizer(b2):
    w, g = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    return w, g, AdamW([w], [g], lr=1e-3, betas=(0.9, b2), state_bits=8)


def _states(opt):
    """m and v in float64."""
    m = opt.m[0].view(torch.float8_e4m3fn).double().view(-1, BLOCK) * opt.m_scale[0].double()[:, None]
    r = opt.v[0].view(torch.float8_e4m3fn).double().view(-1, BLOCK) * opt.v_scale[0].double()[:, None]
    return m, r * r


@pytest.mark.parametrize("b2,steps", [(0.95, 600), (0.999, 14000)])
def test_states_follow_when_only_a_blocks_largest_element_keeps_its_gradient(b2, steps):
    w, g, opt = _optimizer(b2)
    g.fill_(1.0)
    v = 0.0
    for k in range(steps):
        if k == 50:
            g.fill_(0.01)
            g.view(-1, BLOCK)[:, 0] = 1.0
        opt.step()
        v = b2 * v + (1 - b2) * (1.0 if k < 50 else 1e-4)
    ratio = _states(opt)[1][:, 1:] / v
    assert abs(float(ratio.mean()) - 1) <= 0.14 * SIGMA6, float(ratio.mean())
    assert float((ratio - 1).square().mean().sqrt()) <= 0.14 + 0.01


@pytest.mark.parametrize("b2,steps", [(0.95, 600), (0.999, 4000)])
def test_states_of_random_gradients_have_no_bias(b2, steps):
    w, g, opt = _optimizer(b2)
    gen = torch.Generator(device="cuda").manual_seed(7)
    m, v = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
    for _ in range(steps):
        g.normal_(mean=0.3, generator=gen)
        opt.step()
        m.lerp_(g.double(), 1 - 0.9)
        v.lerp_(g.double().square(), 1 - b2)
    got_m, got_v = _states(opt)
    assert abs(float(got_v.sum() / v.sum()) - 1) <= 0.57 * SIGMA6, float(got_v.sum() / v.sum())
    scale = float(m.square().mean().sqrt() / m.mean())
    assert abs(float(got_m.sum() / m.sum()) - 1) <= 0.15 * scale * SIGMA6, float(got_m.sum() / m.sum())


def test_a_weight_without_gradients_comes_to_rest():
    """m of elements whose gradients stop falls to zero beside one that goes
    on (229376 smallest codes times 0.9^400 are expected to be left: 10^-13)."""
    w, g, opt = _optimizer(0.95)
    g.fill_(1.0)
    for _ in range(20):
        opt.step()
    g.zero_()
    g.view(-1, BLOCK)[:, 0] = 1.0
    for _ in range(400):
        opt.step()
    assert (_states(opt)[0][:, 1:] == 0).all()
    rest = w.clone()
    opt.step()
    moved = (w != rest).view(-1, BLOCK)
    assert moved[:, 0].all() and not moved[:, 1:].any()


def _unbiased_plan(T):
    return mx.mx_adamw_plan(T.w, T.g, T.m, T.v, masters=T.master, m_scales=T.ms, v_scales=T.vs, weight_decay=T.decay,
                            unbiased=True)


@pytest.mark.parametrize("weights,grad", [("fp32", "fp32"), ("master", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("gap", [0, 1])
def test_one_step_takes_neighbouring_codes(weights, grad, gap):
    T = Tensors(weights, grad, True, gap=gap)
    R = Tensors(weights, grad, True, gap=gap)
    before = T.values()
    mx.mx_adamw(_unbiased_plan(T), _steps(7), lr=1e-2, beta2=0.95)
    mx.mx_adamw(R.plan, _steps(7), lr=1e-2, beta2=0.95)
    # off by the rounding alone, in units of the gap: within [-1, 1], mean 0, variance at most 1/4
    # (v: of the squares; but for values below the smallest code, which never fall to 0)
    off, slack, total = [0.0, 0.0], [0.0, 0.0], [0, 0]
    for i, (w, m, v, g) in enumerate(before):
        n = w.numel()
        # what comes before the rounding of the codes is what rounding to nearest has
        for a, b in ((T.w, R.w), (T.master, R.master), (T.ms, R.ms), (T.vs, R.vs)):
            assert a[i] is None or torch.equal(a[i], b[i])
        m_ref, m_mag = 0.9 * m + 0.1 * g, 0.9 * m.abs() + 0.1 * g.abs()
        r_ref = (0.95 * v + 0.05 * g * g).sqrt()
        for k, (x, mag, codes, scale) in enumerate(((m_ref, m_mag, T.m[i], T.ms[i]), (r_ref, r_ref, T.v[i], T.vs[i]))):
            s = scale.double().cpu().repeat_interleave(BLOCK)[:n]
            y, near = x / s, 16 * U * (x.abs() + mag) / s
            step = torch.exp2(torch.floor(torch.log2((y.abs() + near).clamp_min(2.0 ** -6))) - 3)
            c = codes.double().cpu()
            _check(c, y, step + near, "codes")
            lo = torch.floor(y / step) * step
            gap, err, room = step, c - y, near
            if k == 1:
                gap, err, room = (lo + step) ** 2 - lo ** 2, c * c - y * y, 2 * (y + near) * near
            some = (y >= 2.0 ** -8) if k == 1 else torch.ones_like(y, dtype=torch.bool)
            off[k] += float((err / gap)[some].sum())
            slack[k] += float((room / gap)[some].sum())
            total[k] += int(some.sum())
    for k in range(2):
        assert total[k] > 30000
        assert abs(off[k]) <= 3 * math.sqrt(total[k]) + slack[k] + total[k] * 2.0 ** -16, (off, total)


def test_the_same_step_gives_the_same_bits_in_any_list_and_another_step_others():
    def run(done, order):
        T = Tensors("master", "bf16", True, sizes=[5000, 300, 70000])
        pick = [[c[i] for i in order] for c in (T.w, T.g, T.m, T.v, T.master, T.ms, T.vs)]
        plan = mx.mx_adamw_plan(*pick[:4], masters=pick[4], m_scales=pick[5], v_scales=pick[6], unbiased=True)
        mx.mx_adamw(plan, _steps(done), lr=1e-2)
        return T

    a, b, c = run(7, [0, 1, 2]), run(7, [2, 0, 1]), run(8, [0, 1, 2])
    for x, y, z in zip(a.m + a.v, b.m + b.v, c.m + c.v):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert not torch.equal(x.view(torch.uint8), z.view(torch.uint8))


def test_zeros_nan_and_infinities():
    """Zeros stay zeros, values on a code stay there, and a NaN or infinity
    reaches its element or block as it does to nearest."""
    T = Tensors("fp32", "fp32", True, sizes=[4 * BLOCK], fresh=True)
    g = torch.zeros(4 * BLOCK)
    g[BLOCK:2 * BLOCK] = 2.0 ** torch.arange(BLOCK).remainder(8)
    g[2 * BLOCK + 5], g[2 * BLOCK + 6] = float("nan"), 1.0
    g[3 * BLOCK + 7], g[3 * BLOCK + 8] = float("inf"), 1.0
    T.g[0].copy_(g.cuda())
    mx.mx_adamw(_unbiased_plan(T), _steps(0), lr=1e-2, beta2=0.95)
    c = T.v[0].float().cpu()
    assert (c[:BLOCK] == 0).all() and (T.m[0].float()[:BLOCK] == 0).all()
    # (448 times a power of two is a code; the scaled value is within an ulp or two of it, and leaves it
    # by a whole step with probability 2^-16 at most)
    assert ((c[BLOCK:2 * BLOCK] / (448 * g[BLOCK:2 * BLOCK] / 128) - 1).abs() > 0).sum() <= 1
    nan = c[2 * BLOCK:3 * BLOCK].isnan()
    assert nan[5] and nan.sum() == 1 and c[2 * BLOCK + 6] == 448
    assert c[3 * BLOCK + 7].isnan() or T.vs[0][3].isinf()
    assert (c[3 * BLOCK + 9:] == 0).all()


def test_a_block_of_zeros_keeps_the_smallest_scale():
    T = Tensors("fp32", "fp32", True, sizes=[BLOCK], fresh=True)
    T.g[0].zero_()
    mx.mx_adamw(_unbiased_plan(T), _steps(0), lr=1e-2)
    assert float(T.ms[0]) == float(T.vs[0]) == pytest.approx(TINY / 448, rel=4 * U)
