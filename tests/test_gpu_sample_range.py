"""Sampling at temperatures so small that neighbouring floats are many powers of two apart."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [20.0, 3.0])
@pytest.mark.parametrize("steps", [40, 90, 110, 123, 125, 126.5, 127.2, 127.5, 127.9, 128.5, 200])
def test_the_largest_logit_is_drawn(steps, M):
    """T such that two floats next to each other near the largest logit have weights 2^-steps apart: all others together are below
    700 * 2^-40, so every number from 0.001 to 0.999 draws the largest, whose log q is 0."""
    N, V, K = 16, 700, 4
    T = float(np.float32(np.log2(np.e) * float(np.spacing(np.float32(M))) / steps))
    z = torch.full((N, V), -5.0)
    z[:, 50::90] = float(np.nextafter(np.float32(M), np.float32(0)))
    z[:, 51::90] = float(np.nextafter(np.nextafter(np.float32(M), np.float32(0)), np.float32(0)))
    at = torch.arange(N) * 43 + 1
    z[torch.arange(N), at] = M
    z, u = z.cuda(), torch.tensor([0.001, 0.3, 0.7, 0.999]).repeat(N, 1).cuda()
    row = lambda v, dt=torch.float32: torch.full((N,), v, dtype=dt, device="cuda")  # noqa: E731
    for knobs in ({}, dict(top_p=row(0.9)), dict(top_k=row(300, torch.int32)), dict(top_k=row(300, torch.int32), top_p=row(0.99)),
                  dict(min_p=row(1e-20))):
        o = rh.rl_sample(z, u, temperature=row(T), capacity=N * V if knobs else 0, **knobs)
        assert o.status_bits() == 0
        assert (o.tokens.cpu() == at[:, None]).all(), knobs
        assert float(o.logq.abs().max()) <= 2.0 ** -20, knobs
