"""What the blocks around the experts do on the host, without a GPU: calls
that they refuse.  Their buffers are on the CPU here, and no call reaches a
kernel."""
import pytest
import torch

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
