"""The training step as a whole: the bf16 layer's outputs and gradients
against autograd in float64, the optimizer's step, checkpoint and captured
replay, and the example, which has to learn."""
import os
import sys

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from mxfp8_block_scaled_04_amd.bf16_layer import Bf16Layer
from mxfp8_block_scaled_04_amd.optimizer import AdamW

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

SIZES, H, I = [70, 0, 131, 1, 54], 64, 96


def _layer(fp32):
    gen = torch.Generator().manual_seed(0)
    M, G = sum(SIZES), len(SIZES)
    off = torch.tensor([sum(SIZES[:g]) for g in range(G + 1)], dtype=torch.int32, device="cuda")
    X, dY = (torch.randn((M, H), generator=gen).bfloat16() for _ in range(2))
    W1 = (torch.randn((G, 2 * I, H), generator=gen) * H ** -0.5).bfloat16()
    W2 = (torch.randn((G, H, I), generator=gen) * I ** -0.5).bfloat16()
    return Bf16Layer(off, M, H, I, fp32_grads=fp32), X, dY, W1, W2


def _reference(X, dY, W1, W2):
    """Float64, no intermediate rounding."""
    X, W1, W2 = (t.double().requires_grad_() for t in (X, W1, W2))
    ys, at = [], 0
    for g, n in enumerate(SIZES):
        p = (X[at:at + n] @ W1[g].t()).reshape(n, I // 32, 2, 32)
        h = torch.nn.functional.silu(p[:, :, 0]) * p[:, :, 1]
        ys.append(h.reshape(n, I) @ W2[g].t())
        at += n
    Y = torch.cat(ys)
    Y.backward(dY.double())
    return Y.detach(), X.grad, W1.grad, W2.grad


def _near(got, ref):
    # bf16 intermediates (preact, h, dh, d(gate, up)): each a relative rounding of at most 2^-8,
    # a handful of them behind every result, averaging over the sums
    err = float((got.double().cpu() - ref).norm() / ref.norm())
    assert err < 4 * 2.0 ** -8, err


@pytest.mark.parametrize("fp32", [False, True])
def test_layer_against_autograd(fp32):
    layer, X, dY, W1, W2 = _layer(fp32)
    dev = [t.cuda() for t in (X, dY, W1, W2)]
    Y, dX, dW1, dW2 = _reference(X, dY, W1, W2)
    _near(layer.forward(dev[0], dev[2], dev[3]), Y)
    for got, ref in zip(layer.backward(*dev), (dX, dW1, dW2)):
        _near(got, ref)
    assert (layer.dW1[1] == 0).all() and (layer.dW2[1] == 0).all()  # the expert without rows
    if fp32:
        once = layer.dW1.clone()
        layer.backward(*dev, accumulate=True)
        assert torch.equal(layer.dW1, once + once)  # x + x is exact


@pytest.mark.parametrize("bits", [32, 8])
def test_checkpoint_resumes_bit_for_bit(bits):
    def make():
        gen = torch.Generator().manual_seed(1)
        ws = [torch.randn(n, generator=gen).bfloat16().cuda() for n in (1000, 256, 3)]
        gs = [torch.randn(n, generator=gen).cuda() for n in (1000, 256, 3)]
        return ws, gs, AdamW(ws, gs, lr=1e-2, weight_decay=[0.1, 0.0, 0.0], state_bits=bits, max_norm=1.0)

    ws, gs, a = make()
    for _ in range(3):
        a.step()
    saved = a.state_dict()
    for _ in range(2):
        a.step()
    ws2, _, b = make()
    b.load_state_dict(saved)
    for _ in range(2):
        b.step()
    assert a.steps.tolist() == b.steps.tolist() == [5, 0]
    assert all(torch.equal(x, y) for x, y in zip(ws, ws2))
    with pytest.raises(ValueError):
        b.load_state_dict({k: v for k, v in saved.items() if k != "lr"})


def test_optimizer_refusals():
    w, g = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        AdamW([w], [g], state_bits=16)
    with pytest.raises(ValueError):
        AdamW([], [])
    with pytest.raises(ValueError):
        AdamW([w], [g, g])


def test_captured_step_of_layer_and_optimizer():
    """Forward, backward, norm and step captured once; replays equal eager steps bit for bit."""
    def make():
        layer, X, dY, W1, W2 = _layer(True)
        X, dY, W1, W2 = (t.cuda() for t in (X, dY, W1, W2))
        opt = AdamW([W1, W2], [layer.dW1, layer.dW2], lr=1e-2, state_bits=8, max_norm=1.0)

        def step():
            layer.forward(X, W1, W2)
            layer.backward(X, dY, W1, W2)
            opt.step()

        return step, opt, layer

    eager, a, la = make()
    captured, b, lb = make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for k in range(4):
        eager()
        graph.replay()
        torch.cuda.synchronize()
        assert a.steps.tolist() == b.steps.tolist() == [k + 1, 0]
        assert torch.equal(la.y, lb.y) and torch.equal(a.norm, b.norm)
        assert all(torch.equal(x, y) for x, y in zip(a.weights, b.weights))


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns(precision, bits):
    import train_experts

    losses = train_experts.train(precision, bits, steps=40)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.5 * losses[0], losses[::10]
