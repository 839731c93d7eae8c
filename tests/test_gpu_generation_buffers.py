"""The generation operators' own buffers: workspaces with any contents."""
import pytest
import torch

import lm_head_gb300 as rh

pytestmark = pytest.mark.gpu


def sampling_inputs(N=40, V=5000):
    g = torch.Generator().manual_seed(4)
    z = (3 * torch.randn(N, V, generator=g)).cuda()
    top_p = torch.full((N,), 0.9, device="cuda")
    top_p[::3] = 1.0
    return z, torch.rand(N, 5, generator=g).cuda(), top_p


@pytest.mark.parametrize("fill", [0, 1, 255])
def test_a_sampling_workspace_may_hold_anything(fill):
    z, u, top_p = sampling_inputs()
    want = rh.rl_sample(z, u, top_p=top_p, capacity=z.numel())
    n = rh.rl_sample_workspace_bytes(*z.shape, u.shape[1])
    for _ in range(2):          # a workspace that was just used, too
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            o = rh.rl_sample(z, u, top_p=top_p, capacity=z.numel(), ws=ws)
            assert torch.equal(o.offsets, want.offsets) and torch.equal(o.tokens, want.tokens)
            assert torch.equal(o.ids, want.ids) and torch.equal(o.support_logq, want.support_logq)
            assert o.status_bits() == 0
