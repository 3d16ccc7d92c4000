"""The type bit of unbiased 8-bit states, on the CPU: refusals and the
binding's choice."""
import ctypes

import torch

from mxfp8_block_scaled_04_amd import training as T
from test_abi_train import OK, SHAPE, _plan, _row


def test_unbiased_codes_need_8_bit_states():
    eight = {"ms": 0x6000, "vs": 0x7000}
    assert _plan(_row(types=T.STATE_8BIT | T.UNBIASED, **eight))[0] == OK
    assert _plan(_row(types=T.UNBIASED))[0] == SHAPE
    assert _plan(_row(n=0, types=T.UNBIASED, w=None, g=None, m=None, v=None))[0] == SHAPE
    for unknown in (8, 32, 256):
        assert _plan(_row(types=T.STATE_8BIT | unknown, **eight))[0] == SHAPE


def test_the_binding_marks_the_8_bit_tensors_only(monkeypatch):
    monkeypatch.setattr(T, "_same_device", lambda *tensors: None)
    f, c, s = torch.zeros(300), torch.zeros(300, dtype=torch.uint8), torch.zeros(2)

    def types(**kwargs):
        plan = T.mx_adamw_plan([f, f], [f, f], [f, c], [f, c], m_scales=[None, s], v_scales=[None, s], **kwargs)
        entry = ctypes.sizeof(T.AdamwTensor) + 8
        rows = [T.AdamwTensor.from_buffer_copy(bytes(plan.image[i * entry:(i + 1) * entry].tolist())) for i in range(2)]
        return [r.types & 31 for r in rows]

    assert types() == [0, T.STATE_8BIT]
    assert types(unbiased=True) == [0, T.STATE_8BIT | T.UNBIASED]
