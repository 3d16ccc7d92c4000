"""The router on batches: the instances that many tokens take, against the
formulas in float64, the precision of the weights, and that a token's results
are its own."""
import math

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of float32, relative


def reference(logits, k, bias=None, groups=1, kept=None, top=2, score="softmax", renorm=True, scale=1.0):
    """float64, of logits without NaN and infinity (-infinity: a mask); and the rows that float64 does not decide: a score
    is off by its E-term sum's and its quotient's roundings, less than 2^-50 in all, and the formula's equal sums of
    different pairs (0.447 - 0.053 and 0.197 + 0.197, scores 0.197 and biases of 1/4) are in either order then."""
    l = logits.double()
    T, E = l.shape
    kept, open_ = groups if kept is None else kept, l != -math.inf
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        most = l.amax(1, keepdim=True)
        s = torch.where(open_, torch.exp(l - torch.where(most == -math.inf, 0, most)), 0)
        total = s.sum(1, keepdim=True)
        s = torch.where(total == 0, 0, s / total)
    if bias is None and (groups == 1 or top == 1):  # the order is the same
        c = l.clone()
    else:
        c = s + (0 if bias is None else bias.double())
    c[~open_] = -math.inf
    undecided = torch.zeros(T, dtype=torch.bool, device=l.device)
    if groups > 1:
        best = c.reshape(T, groups, -1).sort(dim=2, descending=True).values[:, :, :top]
        pairs = torch.cat([best[:, :, :1], torch.where(best[:, :, 1:] == -math.inf, 0, best[:, :, 1:])], 2)
        best = pairs.sum(2)
        dropped = torch.ones_like(best, dtype=torch.bool)
        dropped.scatter_(1, best.sort(dim=1, descending=True, stable=True).indices[:, :kept], False)
        near = (best[:, :, None] - best[:, None, :]).abs() <= 2.0 ** -48
        other = (pairs[:, :, None] != pairs[:, None, :]).any(3)
        undecided |= (near & other & (dropped[:, :, None] != dropped[:, None, :])).any(2).any(1)
        c = torch.where(dropped[:, :, None], -math.inf, c.reshape(T, groups, -1)).reshape(T, E)
    order = c.sort(dim=1, descending=True, stable=True)
    experts, there = order.indices[:, :k], order.values[:, :k] != -math.inf
    w = torch.where(there, s.gather(1, experts), 0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0, w / total)
    return torch.where(there, experts, -1).to(torch.int32), scale * w, s, undecided


def _near(got, want, rel):
    assert ((got.double() - want).abs() <= want * rel + 2.0 ** -126).all()


def _check(logits, k, scale=2.5, **kw):
    experts, weights, scores = mx.mx_router(logits, k, scale=scale, scores=True, **kw)
    kw["kept"], kw["top"] = kw.pop("groups_kept", None), kw.pop("group_top", 2)
    e, w, s, undecided = reference(logits, k, scale=scale, **kw)
    assert int(undecided.sum()) <= len(logits) // 20  # (only rows of few distinct logits have such sums)
    assert torch.equal(experts[~undecided], e[~undecided])
    # the sum of E exponentials in any order: E / 8 terms in a row at most, and 16 roundings besides
    rel = U * (16 + logits.shape[1] / 8)
    _near(scores, s, rel)
    # ratios of float64 scores, and sigmoids, are rounded once (2^-40: the reference's own and the kernel's float64)
    _near(weights[~undecided], w[~undecided], U + 2.0 ** -40 if kw.get("renorm", True) or kw["score"] == "sigmoid" else rel)


# (tokens, experts, choices, groups, kept) -> (lanes of a token, experts a lane)
BATCHES = [
    (8193, 16, 4, 4, 2),      # 8, 2
    (8193, 24, 2, 3, 2),      # 8, 4
    (8201, 40, 4, 1, 1),      # 8, 8
    (16411, 60, 4, 3, 2),     # 8, 16
    (16411, 128, 4, 8, 3),    # 8, 16
    (8193, 24, 8, 2, 1),      # 16, 2
    (8193, 64, 8, 1, 1),      # 16, 4
    (8201, 96, 8, 4, 2),      # 16, 8
    (8193, 165, 6, 3, 2),     # 16, 16
    (16411, 256, 8, 8, 4),    # 16, 16
    (16411, 256, 8, 1, 1),    # 16, 16
    (8193, 24, 12, 2, 2),     # 32, 1
    (8193, 60, 16, 4, 2),     # 32, 2
    (8191, 165, 6, 3, 2),     # 32, 8
    (8201, 192, 16, 3, 2),    # 32, 8
    (8193, 512, 10, 4, 2),    # 32, 16
    (16411, 512, 16, 1, 1),   # 32, 16
    (8193, 128, 40, 2, 2),    # 64, 2
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,groups,kept", BATCHES)
def test_batches(T, E, k, groups, kept, kind, score):
    gen = torch.Generator(device="cuda").manual_seed(T + E + k)
    l = (torch.randn((T, E), generator=gen, device="cuda") * 2).to(kind)
    bias = torch.randn(E, generator=gen, device="cuda") * 0.3
    how = {"groups": groups, "groups_kept": kept, "score": score}
    for b in (None, bias):
        for renorm in (True, False):
            _check(l, k, bias=b, renorm=renorm, **how)
    _check(l, k, bias=bias, group_top=1, **how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,kept", BATCHES)
def test_batches_of_ties_and_masks(T, E, k, groups, kept, score):
    """Rows whose candidates do not fit the list of a token at once, next to others."""
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    l = torch.randint(-2, 3, (T, E), generator=gen, device="cuda").float()
    l[::5] = 0.0
    l[1::5] = torch.randn((len(l[1::5]), E), generator=gen, device="cuda")
    l[2::5] += torch.where(torch.rand((len(l[2::5]), E), generator=gen, device="cuda") < 0.8, -math.inf, 0.0)
    l[7] = -math.inf
    bias = torch.randint(-1, 2, (E,), generator=gen, device="cuda").float() / 4
    for b in (None, bias):
        _check(l, k, bias=b, groups=groups, groups_kept=kept, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,step", [(60, 4, 2.0 ** -22), (128, 4, 2.0 ** -21), (256, 8, 2.0 ** -22), (512, 10, 2.0 ** -20)])
def test_batches_of_choices_a_few_float32_steps_apart(E, k, step, score):
    """The bias cancels the scores of every other token and orders its experts by steps that are near what sums in float32
    are off."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn((16411, E), generator=gen, device="cuda") * 2
    l[::2] = l[0]
    s = reference(l[:1], k, score=score)[2][0]
    bias = (0.25 - s + step * torch.randperm(E, generator=gen, device="cuda")).float()
    for groups in (1, 4):
        _check(l, k, bias=bias, groups=groups, groups_kept=max(1, groups // 2), score=score, renorm=False)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(64, 32, 8), (16, 128, 4), (8201, 40, 4), (16411, 256, 8), (8193, 512, 10)])
def test_a_token_does_not_depend_on_its_neighbours(T, E, k, kind):
    """Softmax scores, and weights that are such as they are: the same bits beside tokens of ties, of masks and of ordinary logits."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn((T, E), generator=gen, device="cuda").to(kind)
    bias = torch.randn(E, generator=gen, device="cuda") * 0.1
    ties, masks = l.clone(), l.clone()
    some = torch.rand(T, generator=gen, device="cuda") < 0.3
    ties[some] = 1.0
    masks[some] = torch.where(torch.rand((T, E), generator=gen, device="cuda") < 0.9, -math.inf, 0.0).to(kind)[some]
    for b in (None, bias, bias * 0):
        for groups in (1, 4):
            how = {"bias": b, "groups": groups, "groups_kept": max(1, groups // 2), "renorm": False}
            want = mx.mx_router(l, k, scores=True, **how)
            for other in (ties, masks):
                got = mx.mx_router(other, k, scores=True, **how)
                assert all(torch.equal(a[~some], b[~some]) for a, b in zip(got, want))
