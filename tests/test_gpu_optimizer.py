"""optimizer.AdamW on a module's parameters: backward, step, checkpoint, resume."""
import pytest
import torch

from mxfp8_block_scaled_04_amd.optimizer import AdamW

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_are_trained_and_resume(bits):
    gen = torch.Generator().manual_seed(0)
    x, init = torch.randn((64, 40), generator=gen).cuda(), torch.randn((24, 40), generator=gen)

    def make():
        layer = torch.nn.Linear(40, 24, bias=False, device="cuda")
        with torch.no_grad():
            layer.weight.copy_(init)
        layer.weight.grad = torch.zeros_like(layer.weight)
        return layer, AdamW(list(layer.parameters()), [layer.weight.grad], lr=1e-2, state_bits=bits, max_norm=1.0)

    layer, opt = make()
    losses, grads = [], []
    for k in range(15):
        layer.weight.grad.zero_()
        loss = layer(x).square().mean()
        loss.backward()  # into the gradient that is there
        grads.append(layer.weight.grad.clone())
        opt.step()
        losses.append(float(loss.detach()))
        if k == 9:
            saved = opt.state_dict()
    assert losses == sorted(losses, reverse=True)
    resumed, opt = make()
    opt.load_state_dict(saved)
    for g in grads[10:]:
        resumed.weight.grad.copy_(g)
        opt.step()
    assert torch.equal(layer.weight, resumed.weight) and resumed.weight.requires_grad
