"""The norm's sums over many waves."""
import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
U = 2.0 ** -24  # half a step of float32, relative

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,small", [(16384, 1.375 * 2.0 ** -13), (32768, 0.96875 * 2.0 ** -13)])
def test_small_waves_beside_a_large_one(N, small):
    """One wave's part of the sum is 512, the 15 others' 0.94 of half a step of it each."""
    x = torch.full((3, N), small, dtype=torch.bfloat16, device="cuda")
    x[:, :512] = 1.0
    rstd = mx.mx_rms_norm(x, torch.ones(N, device="cuda"), eps=0.0, y=None, rstd=True)[4]
    want = 1 / x.double().square().mean(1).sqrt()
    # joined in pairs at most two such parts meet the large one alone, and 3 roundings are below half a step: 3 half steps
    # of the sum, half of that in r; the mean is exact, the square root and the quotient are half a step off each
    assert ((rstd.double() - want).abs() <= want * U * (1.5 + 2)).all()
