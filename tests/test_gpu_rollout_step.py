"""The generation operators together (examples/rollout_step.py): a rollout of grouped samples over
a paged cache, then the head's training step on what it recorded.

The trainer's log-probabilities come from the same hidden rows and head weights as the sampler's,
so they agree to the rounding of two fp32 contractions (the bar of the head's own parity
tests, 1e-5 plus accumulation), and the sampler's support carries the masses it claims."""
import os
import sys

import pytest
import torch

import lm_head_gb300 as rh

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_rollout_and_training_step_agree():
    import rollout_step as ex
    policy = ex.Policy.random()
    g = torch.Generator().manual_seed(9)
    prompts = [torch.randint(0, 4096, (n,), generator=g).tolist() for n in (1, 16, 77, 200)]
    r = ex.rollout(policy, prompts, samples=6, steps=20)
    N = r.tokens.numel()
    assert int(r.status.item()) == 0 and N == 4 * 6 * 20
    rep = r.replayed.bool()
    assert bool(rep[0::2].all()) and not bool(rep[1::2].any())
    fwd, dX, dW = ex.train_step(policy, r, torch.randn(N, generator=g).cuda())
    assert fwd.status_bits() == 0, rh.status_names(fwd.status_bits())
    # log P of the label against log q
    assert float((fwd.logp_label - r.logq).abs().max()) < 1e-4
    assert float((fwd.logp_support - r.support_logq).abs().max()) < 1e-4
    m = fwd.metrics()
    assert m["n_rl"] == N and m["masked"] == 0 and abs(m["mismatch_kl"]) / N < 1e-5
    assert bool(torch.isfinite(dX).all()) and bool(torch.isfinite(dW).all())


def test_attention_over_the_cache_equals_attention_over_the_sequence():
    """The paged decode of one sample against plain causal attention over prompt and sample."""
    import rollout_step as ex
    policy = ex.Policy.random(seed=3)
    prompt = [7, 99, 1234, 5, 40, 4000, 77]
    r = ex.rollout(policy, [prompt], samples=2, steps=33)
    toks = r.tokens.view(33, 2)
    for s in range(2):
        seq = torch.cat([torch.tensor(prompt, device="cuda"), torch.tensor([prompt[-1]], device="cuda"), toks[:-1, s].long()])
        q, k, v = (x.double() for x in policy.qkv(seq))
        k, v = (x.repeat_interleave(policy.Hq // policy.Hkv, 1) for x in (k, v))
        a = torch.einsum("qhd,khd->hqk", q, k) / policy.D ** 0.5
        a = a.masked_fill(torch.ones(len(seq), len(seq), device="cuda").triu(1).bool(), float("-inf"))
        o = torch.einsum("hqk,khd->qhd", torch.softmax(a, 2), v).reshape(len(seq), -1)[len(prompt):]
        want = policy.embed[seq[len(prompt):]].double() + o
        got = r.hidden.view(33, 2, -1)[:, s].double()
        # the weights', the output's and the sum's roundings to bf16: half a step of each value
        bar = 2.0 ** -8 * (v.abs().max() + o.abs() + want.abs()) + 1e-3
        assert bool(((got - want).abs() <= bar).all())
