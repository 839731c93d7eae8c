"""rl_sample where its sums are longest: rows of up to 2^20 logits whose weights are all alike."""
import numpy as np
import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [(1 << 20) - 1, 1 << 20])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_constant_row_of_the_largest_vocabulary(V, dt):
    """2^20 weights of 1: the largest total there is.  The random numbers lie in the middle of a token's
    share (in 24 bits, so that they are the same in fp32)."""
    z = torch.zeros(2, V, dtype=dt, device="cuda")
    z[1] = -1.5
    u = (np.array([[0, 262144, 524288, (1 << 20) - 2], [1, 128974, 786432, 1047527]]) + 0.5) / (1 << 20)
    for kn in ({}, {"top_p": [0.5, 0.97]}, {"top_k": [700001, V - 1]}, {"min_p": [0.5, 1.0], "top_p": [0.25, 1.0]}):
        check(z, u, **kn)


def test_a_large_temperature_makes_a_flat_row():
    V = 1 << 20
    z = torch.randn(2, V, generator=torch.Generator().manual_seed(3)).cuda()
    check(z, np.array([[0.3, 0.9], [0.0, 0.6]]), temperature=[1e25, 1e25])
