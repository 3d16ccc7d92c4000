"""The blocks around the experts, forward and backward: against the calls they
are made of, against float64 autograd, and captured."""
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from mxfp8_block_scaled_04_amd.moe_block import DenseBlock, MoEBlock

pytestmark = pytest.mark.gpu

T, K, E, H, I = 300, 2, 8, 256, 256
EPS = 1e-6


def _tensors(seed=0, stream=torch.bfloat16, experts=E):
    gen = torch.Generator().manual_seed(seed)

    def make(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen) * scale).to(dtype).cuda()

    return {"x": make(T, H), "residual": make(T, H, scale=2.0, dtype=stream), "norm": 1 + make(H, scale=0.2),
            "gate": make(E, H, scale=H ** -0.5 * 2), "W1": make(experts, 2 * I, H, scale=H ** -0.5),
            "W2": make(experts, H, I, scale=I ** -0.5), "dout": make(T, H), "dh": make(T, H, dtype=stream),
            "bias": make(E, scale=0.05, dtype=torch.float32)}


def _experts(y, W1, W2):
    """One expert's SwiGLU layer of rows y, float64."""
    p = (y @ W1.t()).reshape(len(y), I // 32, 2, 32)
    return (torch.nn.functional.silu(p[:, :, 0]) * p[:, :, 1]).reshape(len(y), I) @ W2.t()


def _norm(t):
    h = t["x"] + t["residual"]
    return h, h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * t["norm"]


def _near(got, want, limit):
    err = float((got.double().cpu() - want).norm() / want.norm())
    assert err < limit, err


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score,renorm,groups,with_bias", [("softmax", True, 1, False), ("sigmoid", True, 4, True),
                                                           ("softmax", False, 2, True)])
def test_moe_block(score, renorm, groups, with_bias, stream):
    t = _tensors(1, stream)
    bias = t["bias"] if with_bias else None
    block = MoEBlock(T, K, E, H, I, score=score, renorm=renorm, scale=1.5, groups=groups,
                     groups_kept=max(1, groups // 2), stream_dtype=stream, eps=EPS)
    block.quantize_weights(t["W1"], t["W2"])
    out, h = block.forward(t["x"], t["residual"], t["norm"], t["gate"], bias)
    grads = block.backward(t["dout"], t["dh"], t["norm"], t["gate"])

    # the calls it is made of
    y, h2, _, _, rstd = mx.mx_rms_norm(t["x"], t["norm"], residual=t["residual"], eps=EPS, rstd=True)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    logits = mx.mx_grouped_gemm_bf16(y, t["gate"].unsqueeze(0), off)
    how = {"score": score, "renorm": renorm, "scale": 1.5}
    experts, weights, _ = mx.mx_router(logits, K, bias=bias, groups=groups, groups_kept=max(1, groups // 2), **how)
    assert torch.equal(h, h2) and torch.equal(block.experts, experts) and torch.equal(block.weights, weights)
    dweights = mx.mx_combine_dweights(t["dout"], block.routed.layer.y, block.routed.slot_of)
    dlogits = mx.mx_router_backward(logits, experts, dweights, **how)
    dy2 = mx.mx_grouped_gemm_bf16_dgrad(dlogits, t["gate"].unsqueeze(0), off)
    dh, _, dnorm = mx.mx_rms_norm_backward(block.routed.dX, h, t["norm"], rstd, dy2=dy2, dh_in=t["dh"],
                                           dweight=torch.float32)
    assert torch.equal(grads[0], dh) and torch.equal(grads[4], dnorm)

    # float64, with the choices made above
    d = {n: v.double().cpu().requires_grad_() for n, v in t.items()}
    h64, y64 = _norm(d)
    l64 = y64 @ d["gate"].t()
    s = torch.sigmoid(l64) if score == "sigmoid" else torch.softmax(l64, 1)
    w = s.gather(1, experts.cpu().long())
    w = 1.5 * (w / w.sum(1, keepdim=True) if renorm else w)
    ref = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        for i in range(K):
            rows = (experts[:, i] == e).nonzero().flatten().cpu()
            if len(rows):
                ref = ref.index_add(0, rows, w[rows, i, None] * _experts(y64[rows], d["W1"][e], d["W2"][e]))
    (ref * d["dout"].detach()).sum().add((h64 * d["dh"].detach()).sum()).backward()
    # operands in E4M3 are 2^-4 off at most, 0.03 on average; two of them in each of the 5 products behind a result
    _near(out, ref.detach(), 0.15)
    _near(grads[0], d["x"].grad, 0.15)
    _near(grads[1], d["W1"].grad, 0.2)
    _near(grads[2], d["W2"].grad, 0.2)
    _near(grads[3], d["gate"].grad, 0.2)
    _near(grads[4], d["norm"].grad, 0.2)
    assert torch.equal(d["x"].grad, d["residual"].grad)


def test_the_gate_gradient_of_the_expert_outputs_that_there_are():
    """The router's own part, exactly: d gate from the block's bf16 expert rows, in float64."""
    t = _tensors(2)
    block = MoEBlock(T, K, E, H, I)
    block.quantize_weights(t["W1"], t["W2"])
    block.forward(t["x"], t["residual"], t["norm"], t["gate"])
    dgate = block.backward(t["dout"], None, t["norm"], t["gate"])[3]
    rows = block.routed.layer.y.double().cpu()[block.routed.slot_of.cpu().long()]
    g = (rows * t["dout"].double().cpu()[:, None]).sum(2)
    l = block.logits.double().cpu().requires_grad_()
    w = torch.softmax(l, 1).gather(1, block.experts.cpu().long())
    ((w / w.sum(1, keepdim=True)) * g).sum().backward()
    want = l.grad.t() @ block.norm.y.double().cpu()
    size = l.grad.abs().t() @ block.norm.y.double().cpu().abs()
    # d logits are rounded to bf16 (2^-8 of each); fp32 sums of T terms
    assert ((dgate.double().cpu() - want).abs() <= size * (2.0 ** -8 + T * 2.0 ** -24)).all()


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_dense_block(stream):
    t = _tensors(3, stream, experts=1)
    block = DenseBlock(T, H, I, stream_dtype=stream, eps=EPS)
    block.quantize_weights(t["W1"], t["W2"])
    out, h = block.forward(t["x"], t["residual"], t["norm"])
    y = mx.mx_rms_norm(t["x"], t["norm"], residual=t["residual"], eps=EPS)[0]
    q, s = mx.mx_quantize_rows(y)
    assert torch.equal(block.layer.x.q, q) and torch.equal(block.layer.x.s, s)
    first = out.clone()
    assert torch.equal(block.layer.forward(y), first)  # the layer alone quantizes the same rows
    grads = block.backward(t["dout"], t["dh"], t["norm"])
    d = {n: v.double().cpu().requires_grad_() for n, v in t.items()}
    h64, y64 = _norm(d)
    ref = _experts(y64, d["W1"][0], d["W2"][0])
    (ref * d["dout"].detach()).sum().add((h64 * d["dh"].detach()).sum()).backward()
    _near(first, ref.detach(), 0.15)
    for got, name in zip(grads, ("x", "W1", "W2", "norm")):
        _near(got, d[name].grad, 0.2)
    serving = DenseBlock(T, H, I, stream_dtype=stream, eps=EPS, training=False)
    serving.quantize_weights(t["W1"], t["W2"])
    assert torch.equal(serving.forward(t["x"], t["residual"], t["norm"])[0], first)


def test_without_a_residual_the_input_is_the_stream():
    t = _tensors(4, torch.float32)
    block = MoEBlock(T, K, E, H, I, stream_dtype=torch.float32)
    block.quantize_weights(t["W1"], t["W2"])
    out, h = block.forward(t["residual"], None, t["norm"], t["gate"])
    assert h is t["residual"]
    y = mx.mx_rms_norm(t["residual"], t["norm"])[0]
    assert torch.equal(block.norm.y, y)
    dh = block.backward(t["dout"], t["dh"], t["norm"], t["gate"])[0]
    assert dh.dtype == torch.float32
    with pytest.raises(ValueError, match="stream"):
        block.forward(t["x"], None, t["norm"], t["gate"])


def test_the_number_of_experts_is_checked():
    with pytest.raises(ValueError, match="multiple of 8"):
        MoEBlock(T, K, 12, H, I)


def test_two_blocks_captured_and_replayed():
    """A dense and a routed block one after the other, forward and backward."""
    t, u = _tensors(5, experts=1), _tensors(6)
    inputs = [t["x"], t["residual"]]

    def make():
        first, second = DenseBlock(T, H, I), MoEBlock(T, K, E, H, I, score="sigmoid")
        first.quantize_weights(t["W1"], t["W2"])
        second.quantize_weights(u["W1"], u["W2"])

        def step():
            a, h = first.forward(*inputs, t["norm"])
            out, h = second.forward(a, h, u["norm"], u["gate"], u["bias"])
            g2 = second.backward(u["dout"], u["dh"], u["norm"], u["gate"])
            g1 = first.backward(g2[0], g2[0], t["norm"])  # the sum's gradient is that of both
            return [out, h, *g2, *g1]
        return step

    eager, captured = make(), make()
    captured()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = captured()
    for seed in range(3):
        fresh = _tensors(10 + seed)
        inputs[0].copy_(fresh["x"])
        inputs[1].copy_(fresh["residual"])
        want = eager()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
