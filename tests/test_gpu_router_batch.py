"""A token's results are its own, whatever tokens are beside it."""
import math

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx

pytestmark = pytest.mark.gpu


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
