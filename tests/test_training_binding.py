"""What the binding of the training step does on the host, without a GPU: the
stream whose pool a call's own buffers come from, and how a plan's memory is
made.  The library is replaced by a stub that launches nothing."""
import contextlib

import pytest
import torch

from mxfp8_block_scaled_04_amd import training as T


class _Lib:
    """Accepts every call; the sizes are made up."""

    def __getattr__(self, name):
        sizes = {"mx_grouped_gemm_bf16_wgrad_workspace_bytes": 64, "mx_grad_norm_workspace_bytes": 48,
                 "mx_adamw_plan_bytes": 100}
        return lambda *args: sizes.get(name, 0)


@pytest.fixture
def made(monkeypatch):
    """[(shape, stream it was made under)] of every torch.empty of the calls."""
    log, under = [], [None]
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        before = under[0]
        under[0] = s if s is not None else before
        yield
        under[0] = before

    def recorded(*args, **kwargs):
        t = empty(*args, **kwargs)
        log.append((tuple(t.shape), under[0]))
        return t

    monkeypatch.setattr(T, "_lib", lambda: _Lib())
    monkeypatch.setattr(T, "_same_device", lambda *tensors: None)
    monkeypatch.setattr(T, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    return log


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _plan():
    f = [torch.zeros(5)]
    return T.mx_adamw_plan(f, f, f, f)


@pytest.mark.parametrize("side", [None, "another stream"])
def test_buffers_of_a_call_come_from_the_pool_of_its_stream(made, side):
    """Memory of another stream's pool can still be in use there."""
    off = torch.tensor([0, 3], dtype=torch.int32)
    T.mx_grouped_gemm_bf16(_bf16(3, 8), _bf16(1, 16, 8), off, stream=side)
    T.mx_grouped_gemm_bf16_dgrad(_bf16(3, 16), _bf16(1, 16, 8), off, stream=side)
    T.mx_grouped_gemm_bf16_wgrad(_bf16(3, 16), _bf16(3, 8), off, stream=side)
    T.mx_grad_norm(_plan(), stream=side)
    assert [m for m in made if m[0] != (0,)] == [((3, 16), side), ((3, 8), side), ((1, 16, 8), side), ((64,), side),
                                                 ((2,), side)]


def test_the_workspace_of_a_plan_is_zeroed_by_the_plans_own_copy(made, monkeypatch):
    """A fill on the stream that made the plan would not have run yet, or would
    run too late, for a norm on another stream."""
    fills = []
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: fills.append(k.get("device")) or zeros(*a, **k))
    f = [zeros(5)]
    plan = T.mx_adamw_plan(f, f, f, f)
    assert all(d is None for d in fills)  # host memory only
    assert plan.workspace.untyped_storage().data_ptr() == plan.image.untyped_storage().data_ptr()
    assert plan.workspace.numel() == 48 and not plan.workspace.any()
    begin = plan.workspace_address - plan.address
    assert begin >= 100 and begin % 16 == 0 and begin + 48 <= plan.image.numel()
