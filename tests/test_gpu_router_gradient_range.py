"""The gradient of renormalised sigmoid weights where all scores of a token are
small: the weights are ratios of the scores, and so is their gradient."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of float32, relative
LEAST = -709.78271484375  # from this float32 down 1 + e^-l passes the largest float64: S is 0


def _log_sigmoid(l):
    return np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))


def _reference(l, experts, g, scale):
    """(gradient, magnitude of what is added up in it, distance from the largest chosen logit), float64, from logarithms."""
    l, g, at = l.double().cpu().numpy(), g.double().cpu().numpy(), experts.cpu().numpy().astype(int)
    chosen = np.take_along_axis(l, at, 1)
    logs = _log_sigmoid(chosen)
    p = np.exp(logs - logs.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    slope = scale * p * np.exp(_log_sigmoid(-chosen))
    part = slope * (g - (p * g).sum(1, keepdims=True))
    size = np.abs(slope) * (np.abs(g) + (p * np.abs(g)).sum(1, keepdims=True))
    far = chosen.max(1, keepdims=True) - chosen
    out = [np.zeros_like(l) for _ in range(3)]
    for o, v in zip(out, (part, size, far)):
        np.put_along_axis(o, at, v, 1)
    return out


def _check(l, k, scale=1.5, dscores=None, seed=0):
    experts, weights, _ = mx.mx_router(l, k, score="sigmoid", scale=scale)
    g = torch.randn(weights.shape, generator=torch.Generator().manual_seed(seed)).cuda()
    got = mx.mx_router_backward(l, experts, g, dscores=dscores, score="sigmoid", scale=scale)
    want, mag, far = _reference(l, experts, g, scale)
    # fp32: the sums over the choices (k), 40 roundings besides, and half a step of the distance between two logits, which
    # the exponential makes a relative error of the score
    bound = mag * U * (40 + k + 2 * far.max(1, keepdims=True)) + 2.0 ** -126
    bound += np.abs(want) * torch.finfo(l.dtype).eps / 2
    if dscores is not None:  # s (1 - s) of these logits is below 2^-100
        bound += 2.0 ** -90
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err / bound).max()
    return got, weights


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (33, 64, 6), (20, 256, 8), (9, 1000, 33), (3, 4096, 64)])
@pytest.mark.parametrize("shift", [-80.0, -88.0, -95.0, -104.0, -150.0, -300.0, -680.0])
def test_scores_that_float32_does_not_hold(shift, T, E, k, kind):
    gen = torch.Generator().manual_seed(T + E)
    l = (torch.randn((T, E), generator=gen) * 2 + shift).to(kind).cuda()
    got, weights = _check(l, k)
    assert (weights > 0).all() and (got != 0).any(1).all()
    if shift <= -88.0:
        _check(l, k, dscores=torch.randn((T, E), generator=gen).cuda())


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_chosen_logits_on_both_sides_of_zero(kind):
    gen = torch.Generator().manual_seed(5)
    l = (torch.randn((64, 16), generator=gen) * 60).to(kind).cuda()
    for k in (2, 5, 16):
        _check(l, k)


def test_where_the_sum_is_zero_the_gradient_is():
    """As the weights: where every chosen score underflows in float64."""
    l = torch.full((6, 16), -2000.0, device="cuda")
    l[:3, 3] = torch.tensor([np.nextafter(np.float32(LEAST), np.float32(0)), LEAST, -710.5], device="cuda")
    l[3, :4] = -709.0
    experts, weights, _ = mx.mx_router(l, 4, score="sigmoid")
    g = torch.randn((6, 4), generator=torch.Generator().manual_seed(1)).cuda()
    got = mx.mx_router_backward(l, experts, g, score="sigmoid")
    assert (weights != 0).any(1).tolist() == [True, False, False, True, False, False]
    assert (got[[1, 2, 4, 5]] == 0).all()
    assert (got[3, :4] != 0).all() and (got[3, 4:] == 0).all()


@pytest.mark.parametrize("shift", [0.0, -95.0, -300.0])
def test_against_differences_of_the_weights(shift):
    T, E, k = 6, 12, 3
    gen = torch.Generator().manual_seed(2)
    base = torch.linspace(-2, 2, E).repeat(T, 1).gather(1, torch.rand((T, E), generator=gen).argsort(1))
    l = (base + shift).cuda()  # gaps of 0.36: the choice stays
    g = torch.randn((T, k), generator=gen).double().cuda()
    experts = mx.mx_router(l, k, score="sigmoid")[0]
    got = mx.mx_router_backward(l, experts, g.float(), score="sigmoid", scale=1.5)

    def value(l):
        return (mx.mx_router(l, k, score="sigmoid", scale=1.5)[1].double() * g).sum(1)

    h = 2.0 ** -5
    for e in range(E):
        up, down = l.clone(), l.clone()
        up[:, e] += h
        down[:, e] -= h
        diff = (value(up) - value(down)) / (2 * h)
        # third derivatives are at most about as large as the sum of |g|: h^2 / 6 of it; fp32 noise below
        bound = g.abs().sum(1) * 1.5 * (h * h / 6 + 16 * U / h)
        assert ((diff - got[:, e].double()).abs() <= bound).all()
