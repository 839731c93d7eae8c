"""The operators of a speculative rollout together (examples/speculative_rollout.py): drafts, verification, release, fork,
compaction and the drafting model's gradients."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from distill_ref import distill_reference

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def run(seed, steps=8, fork_at=3, drafts=3):
    import rollout_step as base
    import speculative_rollout as ex
    policy = base.Policy.random(seed=seed)
    drafter = ex.Drafter.near(policy)
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(0, 4096, (n,), generator=g).tolist() for n in (1, 16, 77)]
    r = ex.Rollout(policy, drafter, prompts, samples=2, max_new=steps * (drafts + 1), drafts=drafts, seed=seed)
    counts = []
    for i in range(steps):
        counts.append(r.step().accepted.tolist())
        if i == fork_at:
            r.fork()
            live = r.compact()
            lens = r.lens.tolist()
            # a fork shares its full pages: the rows' pages, less one of each pair's full ones, and the prompts'
            full = sum(n // r.page for n, on in zip(lens[::2], r.live[::2]) if on)
            rows = sum(-(-n // r.page) for n, on in zip(lens, r.live) if on)
            assert live == rows - full + sum(-(-len(p) // r.page) for p in prompts)
    return policy, drafter, prompts, r, counts


def hidden_of(policy, seq, n_prompt):
    """The policy's hidden rows of a sequence after its prompt, in 64 bits, and a bar of the paged path's roundings to bf16."""
    seq = torch.tensor(seq, device="cuda")
    q, k, v = (x.double() for x in policy.qkv(seq))
    k, v = (x.repeat_interleave(policy.Hq // policy.Hkv, 1) for x in (k, v))
    a = torch.einsum("qhd,khd->hqk", q, k) / policy.D ** 0.5
    a = a.masked_fill(torch.ones(len(seq), len(seq), device="cuda").triu(1).bool(), float("-inf"))
    o = torch.einsum("hqk,khd->qhd", torch.softmax(a, 2), v).reshape(len(seq), -1)
    want = policy.embed[seq].double() + o
    return want[n_prompt:], (2.0 ** -8 * (v.abs().max() + o.abs() + want.abs()) + 1e-3)[n_prompt:]


def test_rollout_recorded_probabilities():
    """Each row's recorded log-probabilities are the policy's own on its text: whole rows against the softmax of the hidden
    row, to what the hidden row's roundings (half a bf16 step of each value, through the head) allow; truncated ones lie
    above by the mass that was cut, at most log(1 / 0.9)."""
    policy, drafter, prompts, r, counts = run(3)
    assert int(r.status.item()) == 0, rh.status_names(int(r.status.item()))
    assert sum(map(sum, counts)) > 0 and any(c < r.drafts for row in counts for c in row)
    head = policy.head.double()
    for row in range(r.R):
        assert r.live[row] and len(r.texts[row]) == len(r.logqs[row]) and int(r.lens[row]) == len(r.texts[row])
        p = prompts[row // r.per]
        seq = p + [p[-1]] + r.texts[row][:-1]
        h, bar = hidden_of(policy, seq, len(p))
        z = h @ head.T
        lp = torch.log_softmax(z, 1).gather(1, torch.tensor(r.texts[row], device="cuda")[:, None])[:, 0].cpu().numpy()
        got = np.array(r.logqs[row])
        # a logit moves by at most sum |bar| |head|, a log-probability by twice the largest of them
        slack = (2 * (bar @ head.abs().T).amax(1)).cpu().numpy() + 1e-3
        cut = -math.log(0.9) if float(r.top_p[row]) < 1 else 0.0
        assert (got >= lp - slack).all() and (got <= lp + cut + slack).all()
    # forked rows went on by themselves from a common beginning
    same = [a[:4] == b[:4] for a, b in zip(r.texts[::2], r.texts[1::2])]      # (four steps before, a token each at least)
    assert all(same) and any(a != b for a, b in zip(r.texts[::2], r.texts[1::2]))


def test_drafter_gradients():
    """Losses and gradients on the recorded rows against 64 bits: the logits as the call saw them (bf16), so what is left are the
    gradient's rounding to bf16 (2^-8 of each) and the contractions' fp32 sums."""
    import speculative_rollout as ex
    policy, drafter, prompts, r, _ = run(5, steps=4, fork_at=1)
    for kind, tail in (("forward", False), ("reverse", True)):
        loss, dX, dW, x, status = ex.train_step(drafter, r.records, kind, tail, chunk=50)
        assert int(status.item()) == 0
        z = rh.rl_gemm_bf16_tn(x, drafter.head)[0].bfloat16()
        off = np.concatenate([[0], np.cumsum(np.concatenate([np.diff(k.offsets.cpu().numpy()) for k in r.records]))])
        ids, lq = (torch.cat([getattr(k, n) for k in r.records]).cpu().numpy() for n in ("ids", "logq"))
        N = z.shape[0]
        ref = distill_reference(z.float().cpu().numpy(), off, ids, lq, np.full(N, 1.0 / N), kind, tail, 1.0, 0.5)
        assert np.abs(loss.cpu().numpy() - ref["loss"]).max() <= 1e-5 * (1 + np.abs(ref["loss"]).max())
        G = torch.from_numpy(ref["grad"]).cuda()
        xd, hd = x.double(), drafter.head.double()
        bar = 2.0 ** -8 * 1.01 + 1e-5
        assert bool(((dW.double() - G.T @ xd).abs() <= bar * (G.abs().T @ xd.abs()) + 1e-9).all())
        assert bool(((dX.double() - G @ hd).abs() <= bar * (G.abs() @ hd.abs()) + 1e-9).all())


def test_example_runs(capsys):
    import speculative_rollout as ex
    ex.main()
    assert "status []" in capsys.readouterr().out
