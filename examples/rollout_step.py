"""A rollout and one training step on it, with the library's operators from end to end.

Groups of samples are drawn from shared prompts by a policy of one attention layer and an LM
head: per decode step a page plan, the keys and values into the paged cache, attention over
the shared prompt and the sample's own tokens, and sampling that also records each token's log q
and sampler support.  The recorded tokens then go through the head's fused forward and backward.

  python examples/rollout_step.py            # needs the built library and a GB300
"""
from __future__ import annotations

import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lm_head_gb300 as rh  # noqa: E402


@dataclasses.dataclass
class Policy:
    """Random weights of a one-layer policy: embedding, q / k / v projections, LM head."""
    embed: torch.Tensor     # [V, H] bf16
    wqkv: torch.Tensor      # [(Hq + 2 Hkv) D, H] bf16
    head: torch.Tensor      # [V, H] bf16
    Hq: int
    Hkv: int
    D: int

    @staticmethod
    def random(V=4096, H=256, Hq=4, Hkv=2, D=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, k=1.0: (k * torch.randn(*s, generator=g)).bfloat16().cuda()  # noqa: E731
        assert Hq * D == H
        return Policy(r(V, H), r((Hq + 2 * Hkv) * D, H, k=H ** -0.5), r(V, H, k=3 * H ** -0.5), Hq, Hkv, D)

    def qkv(self, tokens):
        x = self.embed[tokens.long()]
        y = (x @ self.wqkv.T).view(-1, self.Hq + 2 * self.Hkv, self.D)
        return y[:, :self.Hq], y[:, self.Hq:self.Hq + self.Hkv], y[:, self.Hq + self.Hkv:]


@dataclasses.dataclass
class Rollout:
    """What the head's loss reads, token by token in decode order."""
    hidden: torch.Tensor
    tokens: torch.Tensor
    logq: torch.Tensor
    offsets: torch.Tensor
    ids: torch.Tensor
    support_logq: torch.Tensor
    replayed: torch.Tensor
    status: torch.Tensor


def rollout(policy: Policy, prompts, samples: int, steps: int, *, page=16, top_p=0.97, temperature=None, draws=16, seed=1):
    """`samples` continuations of `steps` tokens of each prompt (lists of token ids).  Every other
    sample is drawn from its top-p support (replayed later), the others from the whole
    vocabulary with `draws` further draws as their support."""
    dev, i32 = "cuda", torch.int32
    G, R = len(prompts), len(prompts) * samples
    W, WP = -(-steps // page), max(-(-len(p) // page) for p in prompts)
    n_pages = G * WP + R * W
    pool = torch.arange(n_pages, dtype=i32, device=dev)
    cache = [torch.zeros(n_pages, policy.Hkv, page, policy.D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    status = torch.zeros(1, dtype=i32, device=dev)
    t = lambda x: torch.tensor(x, dtype=i32, device=dev)  # noqa: E731

    # the prompts, once per group: their pages, keys and values
    prefix_lens, prefix_table = t([len(p) for p in prompts]), torch.full((G, WP), -1, dtype=i32, device=dev)
    plan = rh.rl_page_plan(prefix_lens, torch.zeros_like(prefix_lens), prefix_table, pool, page_size=page, n_pages=n_pages,
                           n_tokens=sum(map(len, prompts)), status=status)
    _, k, v = policy.qkv(t([x for p in prompts for x in p]))
    rh.rl_kv_append(k, v, plan.slot_map, *cache, status=status)

    group_offsets = t([g * samples for g in range(G + 1)])
    table = torch.full((R, W), -1, dtype=i32, device=dev)
    ones, lens = torch.ones(R, dtype=i32, device=dev), torch.zeros(R, dtype=i32, device=dev)
    used = plan.free_used
    token = t([p[-1] for p in prompts for _ in range(samples)])     # a sample starts from its prompt's last token
    tp = torch.full((R,), top_p, device=dev)
    tp[1::2] = 1.0
    g = torch.Generator(device=dev).manual_seed(seed)
    cap = R * 1024
    got = []
    for _ in range(steps):
        plan = rh.rl_page_plan(ones, lens, table, pool, page_size=page, n_pages=n_pages, n_tokens=R, free_used=used,
                               group_offsets=group_offsets, prefix_lens=prefix_lens, status=status)
        q, k, v = policy.qkv(token)
        rh.rl_kv_append(k, v, plan.slot_map, *cache, status=status)
        a = rh.rl_prefix_attn(q, *cache, plan.cu_q, plan.kv_lens, table, max_q=1, max_kv=steps, group_offsets=group_offsets,
                              prefix_lens=prefix_lens, prefix_table=prefix_table, max_prefix=WP * page, status=status)
        hidden = (policy.embed[token.long()] + a.out.view(R, -1)).contiguous()
        logits, _ = rh.rl_gemm_bf16_tn(hidden, policy.head, status=status)
        o = rh.rl_sample(logits, torch.rand(R, 1 + draws, generator=g, device=dev), top_p=tp, temperature=temperature,
                         capacity=cap, status=status)
        got.append((hidden, o))
        token, lens, used = o.tokens[:, 0].contiguous(), plan.kv_lens, plan.free_used
    nnz = [o.nnz() for _, o in got]
    offsets = [torch.zeros(1, dtype=torch.int64, device=dev)]
    for _, o in got:
        offsets.append(offsets[-1][-1] + o.offsets[1:])
    return Rollout(torch.cat([h for h, _ in got]), torch.cat([o.tokens[:, 0] for _, o in got]),
                   torch.cat([o.logq[:, 0] for _, o in got]), torch.cat(offsets),
                   torch.cat([o.ids[:n] for (_, o), n in zip(got, nnz)]),
                   torch.cat([o.support_logq[:n] for (_, o), n in zip(got, nnz)]),
                   torch.cat([o.replayed for _, o in got]), status)


def train_step(policy: Policy, r: Rollout, adv):
    """The head's loss, metrics and gradients on a rollout (token mean)."""
    N = r.tokens.numel()
    batch = rh.HeadBatch(r.hidden, policy.head, r.tokens, r.logq, adv, r.offsets, r.ids, r.support_logq, r.replayed)
    return rh.rl_head_loss_fwd_bwd(batch, rh.HeadParams(loss_type=rh.RL_LOSS_IPO), torch.full((N,), 1.0 / N, device="cuda"))


def main():
    policy = Policy.random()
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, 4096, (n,), generator=g).tolist() for n in (37, 16, 150, 5)]
    r = rollout(policy, prompts, samples=8, steps=24)
    adv = torch.randn(r.tokens.numel(), generator=g).cuda()
    fwd, dX, dW = train_step(policy, r, adv)
    m = fwd.metrics()
    n = m["n_rl"]
    print(f"status {rh.status_names(int(r.status.item()) | fwd.status_bits())}  tokens {n}  support entries {r.ids.numel()}  "
          f"loss {m['loss'] / n:.5f}  mismatch_kl {m['mismatch_kl'] / n:.2e}  support_mass {m['support_mass'] / n:.4f}  "
          f"|dX| {float(dX.float().norm()):.4f}  |dW| {float(dW.norm()):.4f}")


if __name__ == "__main__":
    main()
