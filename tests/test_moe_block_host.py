"""What the blocks around the experts do on the host, without a GPU: calls
that they refuse.  Their buffers are on the CPU here, and no call reaches a
kernel."""
import types

import pytest
import torch

from mxfp8_block_scaled_04_amd import moe_block as M
from mxfp8_block_scaled_04_amd.moe_block import DenseBlock, MoEBlock

T, K, E, H, I = 6, 2, 8, 256, 256


def _moe(**kw):
    return MoEBlock(T, K, E, H, I, device="cpu", **kw)


def _dense(**kw):
    return DenseBlock(T, H, I, device="cpu", **kw)


def _rows(dtype=torch.bfloat16):
    return torch.zeros((T, H), dtype=dtype)


NORM, GATE = torch.zeros(H, dtype=torch.bfloat16), torch.zeros((E, H), dtype=torch.bfloat16)


def test_a_block_without_training_has_no_backward_pass():
    block = _dense(training=False)
    block.norm.h = _rows()  # (as a forward pass leaves it)
    with pytest.raises(ValueError, match="training=False"):
        block.backward(_rows(), None, NORM)


def test_backward_needs_a_forward_pass():
    with pytest.raises(ValueError, match="forward"):
        _dense().backward(_rows(), None, NORM)
    with pytest.raises(ValueError, match="forward"):
        _moe().backward(_rows(), None, NORM, GATE)


def test_output_gradients_of_other_rows_are_refused():
    """(The first kernel of the backward pass writes as many rows as dout has.)"""
    for block, more in ((_dense(), (NORM,)), (_moe(), (NORM, GATE))):
        block.norm.h = _rows()
        with pytest.raises(ValueError, match="dout must be a matrix of 6 x 256"):
            block.backward(torch.zeros((T + 1, H), dtype=torch.bfloat16), None, *more)
        with pytest.raises(ValueError, match="dout must be a matrix of 6 x 256"):
            block.backward(torch.zeros((T, 2 * H), dtype=torch.bfloat16), None, *more)
        with pytest.raises(TypeError, match="dout must be bfloat16"):
            block.backward(_rows(torch.float32), None, *more)
        with pytest.raises(ValueError, match="contiguous rows"):
            block.backward(torch.zeros((H, T), dtype=torch.bfloat16).t(), None, *more)
        with pytest.raises(ValueError, match="one GPU"):
            block.backward(_rows(), None, *more)


def test_weights_of_another_place_are_refused():
    for block, G in ((_dense(), 1), (_moe(), E)):
        W1, W2 = torch.zeros((G, 2 * I, H), dtype=torch.bfloat16), torch.zeros((G, H, I), dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="one GPU"):
            block.quantize_weights(W1, W2)


def test_every_call_is_made_with_the_blocks_gpu_as_the_current_one(monkeypatch):
    """(The calls of the norm and the router go to their tensors' GPU by themselves, the others to the current one.)"""
    now, log = [0], []

    class _Device:
        def __init__(self, at):
            self.at = at

        def __enter__(self):
            self.before, now[0] = now[0], self.at

        def __exit__(self, *_):
            now[0] = self.before

    def record(name, result=None):
        def call(*args, **kw):
            log.append((name, now[0]))
            return result
        return call

    moe, dense = _moe(), _dense()
    for block in (moe, dense):
        block.norm.y = types.SimpleNamespace(get_device=lambda: 1, shape=(T, H))  # the block is on GPU 1, GPU 0 is current
    monkeypatch.setattr(M, "_current_device", lambda: now[0])
    monkeypatch.setattr(M, "_one_gpu", lambda *tensors: 1)
    monkeypatch.setattr(torch.cuda, "device", _Device)
    for name in [n for n in vars(M) if n.startswith("mx_")]:
        monkeypatch.setattr(M, name, record(name, (None, _rows(), None, None, None)))
    for layer in (moe.routed, moe.routed.layer, dense.layer):
        for name in ("quantize_weights", "forward", "forward_experts", "backward"):
            monkeypatch.setattr(layer, name, record(name, (_rows(), None, None)), raising=False)
    for block, more in ((moe, (NORM, GATE)), (dense, (NORM,))):
        block.quantize_weights(None, None)
        block.forward(_rows(), _rows(), *more)
        block.backward(_rows(), None, *more)
    assert now == [0] and len(log) == 11 + 6 and all(at == 1 for _, at in log), log
    log.clear()
    now[0] = 1
    monkeypatch.setattr(torch.cuda, "device", None)  # (not set again)
    moe.forward(_rows(), _rows(), NORM, GATE)
    assert len(log) == 4
