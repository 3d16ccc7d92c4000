"""The gradient of the combine's weights against float64 and differences."""
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _make(T, k, N, M, seed=0, ldd=None, ldy=None):
    gen = torch.Generator().manual_seed(seed)

    def rows(R, ld):
        whole = torch.full((R, ld or N), float("nan"), dtype=torch.bfloat16)
        whole[:, :N] = torch.randn((R, N), generator=gen).bfloat16()
        return whole.cuda()[:, :N]

    slot = torch.randint(-2, M + 2, (T, k), generator=gen, dtype=torch.int32)
    return rows(T, ldd), rows(M, ldy), slot.cuda()


def _check(dout, y, slot, **kw):
    got = mx.mx_combine_dweights(dout, y, slot, **kw)
    d, rows, s = dout.double().cpu(), y.double().cpu(), slot.cpu().long()
    inside = (s >= 0) & (s < rows.shape[0])
    if rows.shape[0] == 0:
        assert (got == 0).all()
        return got
    prod = d[:, None, :] * rows[s.clamp(0, rows.shape[0] - 1)]
    want, mag = prod.sum(2) * inside, prod.abs().sum(2)
    # products of bf16 values are exact in fp32; a lane adds N / 256 of them in a row (8 at least), the lanes and waves
    # 10 times
    bound = mag * U * (8 + dout.shape[1] / 256 + 10)
    assert ((got.double().cpu() - want).abs() <= bound).all()
    assert (got.cpu()[~inside] == 0).all()
    return got


@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (5, 2, 64), (33, 8, 512), (17, 3, 1480), (9, 9, 2048), (4, 17, 2056),
                                   (300, 2, 7168), (3, 1, 20488), (2, 70, 128)])
def test_against_float64(T, k, N):
    _check(*_make(T, k, N, max(1, T * k // 2)))
    _check(*_make(T, k, N, 7, seed=1, ldd=N + 8, ldy=N + 24))


def test_no_rows_no_columns_no_tokens():
    dout, _, slot = _make(5, 2, 64, 3)
    empty = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    assert (mx.mx_combine_dweights(dout, empty, slot) == 0).all()
    assert mx.mx_combine_dweights(empty, dout, slot[:0]).shape == (0, 2)
    none = torch.zeros((5, 0), dtype=torch.bfloat16, device="cuda")
    assert (mx.mx_combine_dweights(none, none, slot) == 0).all()


def test_rows_without_a_slot_may_hold_anything():
    dout, y, slot = _make(40, 3, 256, 50)
    y[20:] = float("nan")
    slot[slot >= 20] = -1
    got = _check(dout, torch.where(y.isnan(), 0, y), slot)
    out = torch.full((42, 3), 5.0, device="cuda")
    mx.mx_combine_dweights(dout, y, slot, dweights=out[:40])
    assert torch.equal(out[:40], got) and (out[40:] == 5).all()


def test_is_the_gradient_of_the_combine():
    """The combine is linear in its weights: its fp32 sums times dout."""
    dout, y, slot = _make(20, 4, 128, 30)
    got = mx.mx_combine_dweights(dout, y, slot)
    zero = torch.zeros((20, 4), device="cuda")
    for i in range(4):
        one = zero.clone()
        one[:, i] = 1.0
        out = mx.mx_combine(y, slot, one)  # the rows of choice i, exactly
        want = (dout.double() * out.double()).sum(1)
        mag = (dout.double() * out.double()).abs().sum(1)
        assert ((got[:, i].double() - want).abs() <= mag * U * 20).all()


def test_rows_past_2_31_elements():
    ld, R, N = 1 << 26, 40, 264
    wide = [torch.empty(R * ld, dtype=torch.bfloat16, device="cuda").as_strided((R, N), (ld, 1)) for _ in range(2)]
    dout, y, _ = _make(R, 2, N, R)
    slot = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda").reshape(R, 1).repeat(1, 2)
    for w, t in zip(wide, (dout, y)):
        w.copy_(t)
    assert torch.equal(mx.mx_combine_dweights(wide[0], wide[1], slot), _check(dout, y, slot))


def test_same_bits_every_time_and_on_another_stream():
    args = _make(500, 8, 2048, 4000)
    want = mx.mx_combine_dweights(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        got = mx.mx_combine_dweights(*args, stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
