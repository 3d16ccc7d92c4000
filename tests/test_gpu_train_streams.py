"""The training-step calls on a stream other than the one that is current."""
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu


def _tensors(n=70001, seed=0):
    gen = torch.Generator().manual_seed(seed)
    w, g, m, v = (torch.randn(n, generator=gen) for _ in range(4))
    return [t.cuda() for t in (w, g, m, v.square())]


def _busy():
    """Work that keeps the current stream occupied for some milliseconds."""
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        a = a @ a
        a = a / a.norm()
    return a


def test_norm_and_step_right_after_the_plan_was_made_on_a_busy_stream():
    first = _tensors()
    steps = torch.tensor([4, 0], dtype=torch.int64, device="cuda")
    plan = mx.mx_adamw_plan(*([t] for t in first))
    norm = mx.mx_grad_norm(plan, 1.0)
    mx.mx_adamw(plan, steps, lr=1e-2, grad_scale=norm[1:])
    want = float((first[1].double() ** 2).sum().sqrt())
    assert abs(float(norm[0]) - want) <= 2.0 ** -23 * want
    side = torch.cuda.Stream()
    for _ in range(5):
        tensors, again = _tensors(), torch.tensor([4, 0], dtype=torch.int64, device="cuda")
        out = torch.full((2,), -1.0, device="cuda")
        keep = _busy()
        plan = mx.mx_adamw_plan(*([t] for t in tensors))
        keep = _busy()  # the stream that made the plan has more to do; the calls do not wait for it
        mx.mx_grad_norm(plan, 1.0, out=out, stream=side)
        mx.mx_adamw(plan, again, lr=1e-2, grad_scale=out[1:], stream=side)
        side.synchronize()
        assert torch.equal(out, norm) and again.tolist() == [5, 0]
        assert all(torch.equal(a, b) for a, b in zip(tensors, first))
        assert not plan.workspace.view(torch.int64)[-1]  # the ticket, ready for the next call
        del keep


def test_outputs_of_a_call_on_another_stream_are_not_memory_of_the_current_streams_pool():
    off = torch.tensor([0, 400, 1000], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(1)
    x, w, dy = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((1000, 256), (2, 512, 256), (1000, 512)))
    plan = mx.mx_adamw_plan(*([t] for t in _tensors()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls = [lambda s: mx.mx_grouped_gemm_bf16(x, w, off, stream=s),
             lambda s: mx.mx_grouped_gemm_bf16_dgrad(dy, w, off, stream=s),
             lambda s: mx.mx_grouped_gemm_bf16_wgrad(dy, x, off, stream=s), lambda s: mx.mx_grad_norm(plan, stream=s)]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        freed = torch.empty_like(want)
        at = freed.data_ptr()
        del freed  # the block that the current stream's pool gives out next
        got = call(side)
        assert got.data_ptr() != at
        side.synchronize()
        assert torch.equal(got, want)
