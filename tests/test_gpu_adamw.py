"""The AdamW step and the gradient norm against the formulas in float64.

Tolerances.  m and v are three fp32 roundings of terms whose magnitudes are
bounded by the sum of magnitudes of their terms: 4 2^-24 of it.  w is
keep w - size u with u = m / (sqrt(v) root + eps): sqrt, the product and the
quotient are each within 2^-24 of their values, m and v as above (v enters as
its root), the constants within 2^-24 each: 16 2^-24 |size u'|, with u' the
update of |m|'s sum of magnitudes, plus 2 2^-24 |w|.  bf16 weights (8 bits) add half a
step, 2^-8 of the value.  An 8-bit state is within half an E4M3 step of the exact value in
units of its scale: 2^-4 of the value or 2^-10, plus 8 2^-24 of it."""
import math

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu

BLOCK, TINY, U = 256, 2.0 ** -100, 2.0 ** -24
SIZES = [1, 3, 4, 255, 256, 257, 1000, 4095, 4096, 4097, 20000, 0, 5]


def _codes(x):
    """x in whole blocks -> (E4M3 values as float64 in units of the scale, scale)."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    amax = b.abs().amax(1).clamp_min(TINY)
    return (b * (448.0 / amax)[:, None]).float().to(torch.float8_e4m3fn).view(-1)[:n], (amax / 448.0).float()


class Tensors:
    """A list of tensors of every size on the GPU, and their values in float64."""

    def __init__(self, weights, grad, eight, sizes=SIZES, seed=0, gap=0, gscale=1.0, fresh=False):
        gen = torch.Generator().manual_seed(seed)
        self.weights, self.eight, self.sizes = weights, eight, sizes
        self.w, self.master, self.g, self.m, self.v, self.ms, self.vs = ([] for _ in range(7))
        self.decay = [0.1 * (i % 3) for i in range(len(sizes))]

        def put(t):  # `gap` elements past a 16-byte boundary
            full = torch.empty(t.numel() + gap, dtype=t.dtype, device="cuda")
            part = full[gap:]
            part.view(torch.uint8).copy_(t.view(torch.uint8))
            return part

        for n in sizes:
            w = torch.randn(n, generator=gen)
            g = torch.randn(n, generator=gen) * gscale * 10.0 ** torch.randint(-3, 1, (n,), generator=gen)
            m = torch.zeros(n) if fresh else torch.randn(n, generator=gen) * 0.1 * gscale
            r = torch.zeros(n) if fresh else torch.randn(n, generator=gen).abs() * 0.3 * gscale
            self.w.append(put(w if weights == "fp32" else w.bfloat16()))
            self.master.append(put(w) if weights == "master" else None)
            self.g.append(put(g.bfloat16() if grad == "bf16" else g))
            if eight:
                (mc, ms), (vc, vs) = _codes(m), _codes(r)
                if fresh:
                    ms, vs = torch.zeros_like(ms), torch.zeros_like(vs)
                self.m.append(put(mc))
                self.v.append(put(vc))
                self.ms.append(ms.cuda())
                self.vs.append(vs.cuda())
            else:
                self.m.append(put(m))
                self.v.append(put(r * r))
        self.plan = mx.mx_adamw_plan(self.w, self.g, self.m, self.v, masters=self.master,
                                     m_scales=self.ms if eight else None, v_scales=self.vs if eight else None,
                                     weight_decay=self.decay)

    def values(self):
        """[(w, m, v, g)] in float64 on the CPU."""
        out = []
        for i, n in enumerate(self.sizes):
            w = (self.master[i] if self.weights == "master" else self.w[i]).double().cpu()
            m, v = self.m[i].double().cpu(), self.v[i].double().cpu()
            if self.eight:
                m = m * self.ms[i].double().cpu().repeat_interleave(BLOCK)[:n]
                v = (v * self.vs[i].double().cpu().repeat_interleave(BLOCK)[:n]) ** 2
            out.append((w, m, v, self.g[i].double().cpu()))
        return out


def _check(got, ref, tol, what):
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3], tol[bad][:3])


def _check_step(T, before, t, c=1.0, lr=1e-2, b1=0.9, b2=0.95, eps=1e-8):
    after = T.values()
    for i, ((w, m, v, g), (w2, m2, v2, _)) in enumerate(zip(before, after)):
        g = g * c
        m_ref, v_ref = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        m_mag = b1 * m.abs() + (1 - b1) * g.abs()
        size, root = lr / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
        den = v_ref.sqrt() * root + eps
        w_ref = (1 - lr * T.decay[i]) * w - size * m_ref / den
        tol = 16 * U * size * m_mag / den + 2 * U * (w.abs() + w_ref.abs())
        if T.weights == "bf16":
            tol = tol + 2.0 ** -8 * (w_ref.abs() + tol)
        _check(w2, w_ref, tol, "w")
        if T.weights == "master":
            assert torch.equal(T.w[i].cpu(), T.master[i].cpu().bfloat16())
        if not T.eight:
            _check(m2, m_ref, 4 * U * m_mag, "m")
            _check(v2, v_ref, 4 * U * v_ref, "v")
            continue
        n = w.numel()
        r_ref = v_ref.sqrt()
        for x, mag, codes, scale, what in ((m_ref, m_mag, T.m[i], T.ms[i], "m"), (r_ref, r_ref, T.v[i], T.vs[i], "v")):
            blocks = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
            biggest = torch.nn.functional.pad(mag, (0, -n % BLOCK)).view(-1, BLOCK).abs().amax(1)
            amax = blocks.abs().amax(1).clamp_min(TINY) if n else blocks.new_zeros(0)
            s = amax / 448
            _check(scale.double().cpu(), s, 8 * U * (s + biggest / 448), what + " scale")
            y = x / s.repeat_interleave(BLOCK)[:n]
            near = 8 * U * (y.abs() + (mag / s.repeat_interleave(BLOCK)[:n]))
            if what == "v":
                y = torch.where(x > 0, y.clamp_min(2.0 ** -9), y)
            _check(codes.double().cpu(), y, torch.maximum(2.0 ** -4 * y.abs(), torch.full_like(y, 2.0 ** -10)) + near,
                   what + " codes")


def _steps(n):
    return torch.tensor([n, 0], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("weights", ["fp32", "master", "bf16"])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("gap", [0, 1, 4])
def test_step(weights, grad, eight, gap):
    T = Tensors(weights, grad, eight, gap=gap)
    steps = _steps(7)
    before = T.values()
    mx.mx_adamw(T.plan, steps, lr=1e-2, beta2=0.95)
    _check_step(T, before, 8)
    assert steps.tolist() == [8, 0]
    before = T.values()
    mx.mx_adamw(T.plan, steps, lr=1e-2, beta2=0.95)
    _check_step(T, before, 9)
    assert steps.tolist() == [9, 0]


@pytest.mark.parametrize("eight", [False, True])
def test_first_step_from_zero_states(eight):
    T = Tensors("master", "fp32", eight, fresh=True)
    before, steps = T.values(), _steps(0)
    mx.mx_adamw(T.plan, steps, lr=1e-2, beta2=0.95)
    _check_step(T, before, 1)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, float("inf")])
def test_clipped_step(eight, max_norm):
    T = Tensors("fp32", "bf16", eight)
    before, steps = T.values(), _steps(3)
    out = mx.mx_grad_norm(T.plan, max_norm)
    norm = math.sqrt(sum(float((b[3] ** 2).sum()) for b in before))
    assert abs(float(out[0]) - norm) <= 2 * U * norm
    c = min(1.0, max_norm / norm)
    assert abs(float(out[1]) - c) <= 2 * U * c
    mx.mx_adamw(T.plan, steps, lr=1e-2, beta2=0.95, grad_scale=out[1:])
    _check_step(T, before, 4, c=float(out[1]))
    # the same bits again: the sum's order is fixed
    assert all(torch.equal(mx.mx_grad_norm(T.plan, max_norm), out) for _ in range(3))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("eight", [False, True])
def test_a_step_with_infinite_gradients_is_left_out(bad, eight):
    T = Tensors("master", "fp32", eight)
    T.g[6][17] = bad
    kept = [[t.clone() for t in column if t is not None] for column in (T.w, T.master, T.m, T.v, T.ms, T.vs)]
    steps = _steps(5)
    out = mx.mx_grad_norm(T.plan, 1.0)
    assert not math.isfinite(float(out[0])) and math.isnan(float(out[1]))
    mx.mx_adamw(T.plan, steps, lr=1e-2, grad_scale=out[1:])
    assert steps.tolist() == [5, 0]
    for old, column in zip(kept, (T.w, T.master, T.m, T.v, T.ms, T.vs)):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(old, [t for t in column if t is not None]))
    # a negative factor too; zero is a number: the states decay
    mx.mx_adamw(T.plan, steps, lr=1e-2, grad_scale=torch.tensor([-1.0], device="cuda"))
    assert steps.tolist() == [5, 0]


def test_without_a_factor_a_nan_stays_in_its_element_or_block():
    for eight in (False, True):
        T = Tensors("fp32", "fp32", eight, sizes=[1000])
        T.g[0][300] = float("nan")
        mx.mx_adamw(T.plan, _steps(5), lr=1e-2)
        w, m, v, _ = T.values()[0]
        at = torch.arange(1000) == 300
        assert w[at].isnan().all() and m[at].isnan().all() and v[at].isnan().all()
        assert w[~at].isfinite().all() and m[~at].isfinite().all() and v[~at].isfinite().all()


def test_tiny_and_huge_gradients():
    """Blocks of zeros, of values whose squares underflow, and of one huge
    value among small ones: finite results, and no zero code for v > 0."""
    n = 4 * BLOCK
    T = Tensors("fp32", "fp32", True, sizes=[n], fresh=True)
    g = torch.zeros(n)
    g[BLOCK:2 * BLOCK] = 1e-25
    g[2 * BLOCK:3 * BLOCK] = 1e-6
    g[2 * BLOCK] = 1e6
    g[3 * BLOCK:] = 1e-38
    T.g[0].copy_(g.cuda())
    steps = _steps(0)
    for _ in range(3):
        mx.mx_adamw(T.plan, steps, lr=1e-2)
    w, m, v, _ = T.values()[0]
    assert w.isfinite().all() and m.isfinite().all() and v.isfinite().all()
    assert (m[:BLOCK] == 0).all() and (v[:BLOCK] == 0).all()
    assert (T.v[0].view(torch.uint8)[2 * BLOCK:3 * BLOCK].cpu() >= 1).all()


def test_many_tensors_equal_one_by_one_and_chunk_counts():
    sizes = [1 + (i * 977) % 9000 for i in range(300)]
    A, B = Tensors("master", "bf16", True, sizes=sizes), Tensors("master", "bf16", True, sizes=sizes)
    sa, sb = _steps(2), _steps(2)
    mx.mx_adamw(A.plan, sa, lr=1e-3)
    for i in range(len(sizes)):
        one = mx.mx_adamw_plan(B.w[i:i + 1], B.g[i:i + 1], B.m[i:i + 1], B.v[i:i + 1], B.master[i:i + 1],
                               B.ms[i:i + 1], B.vs[i:i + 1], weight_decay=B.decay[i:i + 1])
        steps = _steps(2)
        mx.mx_adamw(one, steps, lr=1e-3)
    for x, y in ((A.w, B.w), (A.master, B.master), (A.m, B.m), (A.v, B.v), (A.ms, B.ms), (A.vs, B.vs)):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x, y))
    assert sa.tolist() == [3, 0]


def test_mixed_kinds_in_one_plan():
    kinds = [("fp32", "fp32", False), ("master", "bf16", True), ("bf16", "bf16", False), ("master", "fp32", False)]
    parts = [Tensors(*k, seed=i) for i, k in enumerate(kinds)]
    plan = mx.mx_adamw_plan(*[sum((getattr(p, a) for p in parts), []) for a in ("w", "g", "m", "v", "master")],
                            m_scales=sum((p.ms if p.eight else [None] * len(SIZES) for p in parts), []),
                            v_scales=sum((p.vs if p.eight else [None] * len(SIZES) for p in parts), []),
                            weight_decay=sum((p.decay for p in parts), []))
    before = [p.values() for p in parts]
    mx.mx_adamw(plan, _steps(10), lr=1e-2, beta2=0.95)
    for p, b in zip(parts, before):
        _check_step(p, b, 11)


def test_large_count_of_steps_and_lr_on_the_device():
    T = Tensors("fp32", "fp32", False)
    before, steps = T.values(), _steps(1000000)
    lr = torch.tensor([1e-2], device="cuda")
    mx.mx_adamw(T.plan, steps, lr=lr, beta2=0.95)
    _check_step(T, before, 1000001, lr=float(lr.double()))


def test_captured_steps_follow_the_eager_ones():
    A, B = Tensors("master", "bf16", True), Tensors("master", "bf16", True)
    sa, sb = _steps(0), _steps(0)
    lra, lrb, out = torch.tensor([1e-2], device="cuda"), torch.tensor([1e-2], device="cuda"), torch.zeros(2, device="cuda")

    def step(T, steps, lr, out):
        mx.mx_grad_norm(T.plan, 1.0, out=out)
        mx.mx_adamw(T.plan, steps, lr=lr, grad_scale=out[1:])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(A, sa, lra, out)
    other = torch.zeros(2, device="cuda")
    for k in range(4):
        lra.fill_(1e-2 / (k + 1))
        lrb.fill_(1e-2 / (k + 1))
        for a, b in zip(A.g, B.g):
            a.mul_(1.5)
            b.mul_(1.5)
        graph.replay()
        step(B, sb, lrb, other)
        torch.cuda.synchronize()
        assert sa.tolist() == sb.tolist() == [k + 1, 0]
        assert torch.equal(out, other)
        for x, y in ((A.w, B.w), (A.master, B.master), (A.m, B.m), (A.v, B.v), (A.ms, B.ms), (A.vs, B.vs)):
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x, y))


def test_empty_plan():
    plan = mx.mx_adamw_plan([], [], [], [])
    steps = _steps(4)
    out = mx.mx_grad_norm(plan, 1.0)
    mx.mx_adamw(plan, steps, lr=1e-3, grad_scale=out[1:])
    assert out.tolist() == [0.0, 1.0] and steps.tolist() == [5, 0]


def test_8bit_states_follow_a_falling_gradient():
    """The states' scale follows a block's largest value as it decays by less
    than a code's step, so sqrt(v) keeps up with gradients that fall: within
    the code's own error of the exact state after 200 steps."""
    n = 8 * BLOCK
    T = Tensors("fp32", "fp32", True, sizes=[n], fresh=True)
    gen = torch.Generator().manual_seed(3)
    base = torch.rand(n, generator=gen) + 0.5
    v, steps = torch.zeros(n, dtype=torch.float64), _steps(0)
    for k in range(200):
        g = base * (1.0 if k < 50 else 0.1)
        T.g[0].copy_(g.cuda())
        mx.mx_adamw(T.plan, steps, lr=1e-3, beta2=0.95)
        v = 0.95 * v + 0.05 * g.double() ** 2
    got = T.values()[0][2].sqrt()
    assert ((got / v.sqrt() - 1).abs() < 0.15).all()


def test_a_tensor_past_2_31_elements():
    """8-bit states, bf16 weights and gradients, n > 2^31: the blocks at both
    ends and around element 2^31 equal the same blocks stepped by themselves."""
    n = 2 ** 31 + 3 * BLOCK + 5
    gen = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randn(1 << 20, generator=gen, device="cuda").bfloat16()
    reps = -(-n // base.numel())
    w, g = base.repeat(reps)[:n], base.flip(0).repeat(reps)[:n]
    m, v = (torch.randint(1, 100, (1 << 20,), generator=gen, device="cuda", dtype=torch.uint8).repeat(reps)[:n]
            for _ in range(2))
    blocks = -(-n // BLOCK)
    ms, vs = (torch.rand(blocks, generator=gen, device="cuda") * 1e-3 + 1e-6 for _ in range(2))
    parts = []
    for b in (0, 2 ** 31 // BLOCK - 2, 2 ** 31 // BLOCK, blocks - 2):
        e, s = slice(b * BLOCK, min((b + 2) * BLOCK, n)), slice(b, min(b + 2, blocks))
        parts.append((e, s, [t[e].clone() for t in (w, g, m, v)] + [t[s].clone() for t in (ms, vs)]))
    plan = mx.mx_adamw_plan([w], [g], [m], [v], m_scales=[ms], v_scales=[vs], weight_decay=0.1)
    mx.mx_adamw(plan, _steps(3), lr=1e-2)
    for e, s, (pw, pg, pm, pv, pms, pvs) in parts:
        one = mx.mx_adamw_plan([pw], [pg], [pm], [pv], m_scales=[pms], v_scales=[pvs], weight_decay=0.1)
        mx.mx_adamw(one, _steps(3), lr=1e-2)
        assert torch.equal(w[e], pw) and torch.equal(m[e], pm) and torch.equal(v[e], pv)
        assert torch.equal(ms[s], pms) and torch.equal(vs[s], pvs)
    out = mx.mx_grad_norm(plan)
    norm = math.sqrt(sum(float(c.double().square().sum()) for c in g.split(1 << 28)))
    assert abs(float(out[0]) - norm) <= 2 * U * norm


def test_refusals():
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    with pytest.raises(TypeError):
        mx.mx_adamw_plan([f(4).half()], [f(4)], [f(4)], [f(4)])
    with pytest.raises(TypeError):
        mx.mx_adamw_plan([f(4)], [f(4)], [f(4)], [f(4).to(torch.uint8)])
    with pytest.raises(ValueError):
        mx.mx_adamw_plan([f(4)], [f(5)], [f(4)], [f(4)])
    with pytest.raises(ValueError):
        mx.mx_adamw_plan([f(4)], [f(4)], [f(4)], [])
    with pytest.raises(ValueError):
        mx.mx_adamw_plan([f(4, 4)[:, :2]], [f(8)], [f(8)], [f(8)])
    with pytest.raises(mx.MxError):  # 8-bit states need scales
        mx.mx_adamw_plan([f(4)], [f(4)], [f(4).to(torch.uint8)], [f(4).to(torch.uint8)])
    with pytest.raises(mx.MxError):  # masters of float32 weights
        mx.mx_adamw_plan([f(4)], [f(4)], [f(4)], [f(4)], masters=[f(4)])
    plan = mx.mx_adamw_plan([f(4)], [f(4)], [f(4)], [f(4)])
    for bad in ({"beta1": 1.0}, {"beta2": -0.1}, {"eps": -1.0}, {"lr": float("nan")}):
        with pytest.raises(mx.MxError):
            mx.mx_adamw(plan, _steps(0), **{"lr": 1e-3, **bad})
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(mx.MxError):
            mx.mx_grad_norm(plan, bad)
    with pytest.raises(ValueError):
        mx.mx_adamw(plan, torch.zeros(2, device="cuda"), lr=1e-3)
