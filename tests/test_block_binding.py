"""What the binding of the router's and the norm's calls does on the host,
without a GPU: the GPU and the stream that a call is made on, and the stream
whose pool its own buffers come from.  The library is replaced by a stub that
launches nothing."""
import contextlib
import types

import pytest
import torch

from mxfp8_block_scaled_04_amd import block as B


class _Lib:
    def __init__(self, log, now):
        self.log, self.now = log, now

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_bytes"):
                return 64
            self.log.append((name, self.now[0], args[-1]))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """[(entry point, GPU that was current, stream handle)]; tensors are on GPU 1, GPU 0 is current."""
    log, now = [], [0]

    @contextlib.contextmanager
    def device(at):
        before, now[0] = now[0], at
        yield
        now[0] = before

    monkeypatch.setattr(B, "_lib", lambda: _Lib(log, now))
    monkeypatch.setattr(B, "_one_gpu", lambda *tensors: 1)
    monkeypatch.setattr(B, "_current_device", lambda: now[0])
    monkeypatch.setattr(B, "_raw_stream", lambda at: 1000 + at)
    monkeypatch.setattr(torch.cuda, "device", device)
    return log


def _all(stream=None):
    l, x = torch.zeros(3, 8), torch.zeros(3, 8, dtype=torch.bfloat16)
    w, r, i = torch.zeros(8), torch.zeros(3), torch.zeros((3, 2), dtype=torch.int32)
    B.mx_router(l, 2, scores=True, stream=stream)
    B.mx_router_backward(l, i, torch.zeros(3, 2), stream=stream)
    B.mx_combine_dweights(x, x, i, stream=stream)
    B.mx_rms_norm(x, w, residual=l, rstd=True, stream=stream)
    B.mx_rms_norm_backward(x, l, w, r, dx=True, stream=stream)


NAMES = ["mx_router", "mx_router_backward", "mx_combine_dweights", "mx_rms_norm", "mx_rms_norm_backward"]


def test_calls_are_made_on_the_tensors_gpu_and_its_current_stream(calls):
    _all()
    assert calls == [(n, 1, 1001) for n in NAMES]


def test_a_stream_has_to_be_of_the_tensors_gpu(calls, monkeypatch):
    under = []

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "stream", stream)
    mine = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)
    _all(mine)
    assert calls == [(n, 1, 77) for n in NAMES]
    # every buffer of a call's own: router 3, gradient 1, weights 1, norm h, y, rstd, its gradient dh, dx, dweight, workspace
    assert under == [mine] * 12
    with pytest.raises(ValueError, match="another GPU"):
        _all(types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=78))


def test_the_current_gpu_is_not_set_again(calls, monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", None)
    _all()
    assert [c[0] for c in calls] == NAMES


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.uint8])
def test_dweight_has_a_type_that_the_kernels_write(calls, dtype):
    x, w, r = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(8), torch.zeros(3)
    with pytest.raises(TypeError, match="dweight must be bfloat16 or float32"):
        B.mx_rms_norm_backward(x, x, w, r, dweight=dtype)
    with pytest.raises(TypeError, match="dweight must be bfloat16 or float32"):
        B.mx_rms_norm_backward(x, x, w, r, dweight=torch.zeros(8).to(dtype))
    assert calls == []
    for d in (torch.bfloat16, torch.float32):
        assert B.mx_rms_norm_backward(x, x, w, r, dweight=d)[2].dtype is d


def test_numbers_beyond_32_bits_are_refused(calls):
    """(2^32 + 8 experts would be taken for 8.)"""
    many, few = torch.empty((1, 2 ** 32 + 8), device="meta"), torch.zeros(1, 8)
    with pytest.raises(ValueError, match="below 2"):
        B.mx_router(many, 2)
    for kw in ({"groups": 2 ** 32 + 1}, {"groups_kept": 2 ** 32 + 1}, {"group_top": 2 ** 32 + 1}, {"groups": 1 - 2 ** 32}):
        with pytest.raises(ValueError, match="below 2"):
            B.mx_router(few, 2, **kw)
    none = torch.zeros((0, 8))
    with pytest.raises(ValueError, match="below 2"):
        B.mx_router(none, 2 ** 32 + 2)
    i = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="below 2"):
        B.mx_router_backward(many, i, torch.zeros(1, 2))
    with pytest.raises(ValueError, match="below 2"):
        B.mx_combine_dweights(torch.zeros((1, 8), dtype=torch.bfloat16), torch.zeros((1, 8), dtype=torch.bfloat16),
                              torch.empty((1, 2 ** 32 + 2), dtype=torch.int32, device="meta"))
    assert calls == []
    B.mx_router(few, 2, groups=4, groups_kept=2)
    assert [c[0] for c in calls] == ["mx_router"]
