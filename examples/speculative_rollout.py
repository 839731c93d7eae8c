"""A rollout with drafted tokens, branches and page moves, and a training step of the drafting model.

A small drafting model (an embedding and a head) proposes several tokens of each request; the policy
of examples/rollout_step.py runs on them in one step, and verification keeps what the policy's own
sampling would have given.  The pages of what was turned down go back to the pool.  Half-way every
request is forked, and the live pages are moved together.  The drafting model is then trained on the
policy's top tokens at every position that was run.

  python examples/speculative_rollout.py            # needs the built library and a GB300
"""
from __future__ import annotations

import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import lm_head_gb300 as rh  # noqa: E402
from rollout_step import Policy  # noqa: E402


@dataclasses.dataclass
class Drafter:
    """Next-token logits from the last token alone: embedding [V, H] and head [V, H], bf16."""
    embed: torch.Tensor
    head: torch.Tensor

    @staticmethod
    def near(policy: Policy, noise=0.3, seed=7):
        """The policy's own embedding and head, disturbed."""
        g = torch.Generator().manual_seed(seed)
        n = lambda w: (w.float() + noise * w.float().std() * torch.randn(*w.shape, generator=g).cuda()).bfloat16()  # noqa: E731
        return Drafter(n(policy.embed), n(policy.head))

    def logits(self, tokens, status=None):
        return rh.rl_gemm_bf16_tn(self.embed[tokens.long()].contiguous(), self.head, status=status)[0]


@dataclasses.dataclass
class Recorded:
    """One step's rows: the tokens it ran on, and the policy's top tokens after each."""
    tokens: torch.Tensor
    offsets: torch.Tensor
    ids: torch.Tensor
    logq: torch.Tensor


class Rollout:
    """Requests of shared prompts over a paged cache; `texts[r]` is what row r has emitted."""

    def __init__(self, policy: Policy, drafter: Drafter, prompts, samples: int, max_new: int, *, drafts=3, page=16, top_p=0.9, top=32, seed=1):
        self.policy, self.drafter, self.drafts, self.page, self.top = policy, drafter, drafts, page, top
        dev, i32 = "cuda", torch.int32
        self.G, self.per = len(prompts), 2 * samples                # a row of each pair is free until the fork
        self.R = R = self.G * self.per
        self.W, self.WP = -(-(max_new + drafts + 1) // page), max(-(-len(p) // page) for p in prompts)
        self.n_pages = self.G * self.WP + R * self.W
        t = lambda x: torch.tensor(x, dtype=i32, device=dev)  # noqa: E731
        self.pool = torch.randperm(self.n_pages, device=dev).to(i32)
        self.cache = [torch.zeros(self.n_pages, policy.Hkv, page, policy.D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.status = torch.zeros(1, dtype=i32, device=dev)
        self.prompts = prompts
        self.prefix_lens, self.prefix_table = t([len(p) for p in prompts]), torch.full((self.G, self.WP), -1, dtype=i32, device=dev)
        plan = rh.rl_page_plan(self.prefix_lens, torch.zeros_like(self.prefix_lens), self.prefix_table, self.pool, page_size=page,
                               n_pages=self.n_pages, n_tokens=sum(map(len, prompts)), status=self.status)
        _, k, v = policy.qkv(t([x for p in prompts for x in p]))
        rh.rl_kv_append(k, v, plan.slot_map, *self.cache, status=self.status)
        self.used = plan.free_used
        self.groups = t([g * self.per for g in range(self.G + 1)])
        self.table, self.lens = torch.full((R, self.W), -1, dtype=i32, device=dev), torch.zeros(R, dtype=i32, device=dev)
        self.live = [r % 2 == 0 for r in range(R)]
        self.last = t([prompts[r // self.per][-1] for r in range(R)])
        self.top_p = torch.where(torch.arange(R, device=dev) // 2 % 2 == 0, top_p, 1.0).float()      # every other pair truncated
        self.g = torch.Generator(device=dev).manual_seed(seed)
        self.texts, self.logqs, self.records = [[] for _ in range(R)], [[] for _ in range(R)], []

    def u(self, *n):
        return torch.rand(*n, generator=self.g, device="cuda").clamp_(max=1 - 2.0 ** -24)

    def step(self):
        """Drafts, one run of the policy over them, verification, release of the rest."""
        st, k, dev = self.status, self.drafts, "cuda"
        rows = torch.tensor([r for r in range(self.R) if self.live[r]], device=dev)
        n = rows.numel()
        token, drafted, logits = self.last[rows], [self.last[rows]], []
        for _ in range(k):
            logits.append(self.drafter.logits(token, st))
            token = rh.rl_sample(logits[-1], self.u(n, 1), status=st).tokens[:, 0].contiguous()
            drafted.append(token)
        tokens = torch.stack(drafted, 1).reshape(-1).contiguous()           # each request's last token, then its drafts
        # row i of request j was drafted from row i * n + j of the logits (the last has none)
        held = (torch.arange(k + 1, device=dev).clamp(max=k - 1)[None] * n + torch.arange(n, device=dev)[:, None]).reshape(-1)
        draft = rh.Dist(logits=torch.cat(logits), rows=held.to(torch.int32))

        q_lens = torch.zeros(self.R, dtype=torch.int32, device=dev)
        q_lens[rows] = k + 1
        T = n * (k + 1)
        plan = rh.rl_page_plan(q_lens, self.lens, self.table, self.pool, page_size=self.page, n_pages=self.n_pages, n_tokens=T,
                               free_used=self.used, group_offsets=self.groups, prefix_lens=self.prefix_lens, status=st)
        q, key, val = self.policy.qkv(tokens)
        rh.rl_kv_append(key, val, plan.slot_map, *self.cache, status=st)
        a = rh.rl_prefix_attn(q, *self.cache, plan.cu_q, plan.kv_lens, self.table, max_q=k + 1, max_kv=self.W * self.page,
                              group_offsets=self.groups, prefix_lens=self.prefix_lens, prefix_table=self.prefix_table,
                              max_prefix=self.WP * self.page, status=st)
        hidden = (self.policy.embed[tokens.long()] + a.out.view(T, -1)).contiguous()
        z, _ = rh.rl_gemm_bf16_tn(hidden, self.policy.head, status=st)
        # the rows' distributions: truncated ones as support rows, the others whole
        o = rh.rl_sample(z, self.u(T, 1), top_p=self.top_p.repeat_interleave(q_lens), capacity=T * z.shape[1], status=st)
        target = rh.Dist(logits=z, offsets=o.offsets, ids=o.ids, logq=o.support_logq, replayed=o.replayed)
        v = rh.rl_verify(tokens, plan.cu_q, self.u(T), self.u(self.R), target, draft, vocab=z.shape[1], ctx_lens=self.lens, status=st)
        # what the drafting model learns from: the policy's top tokens after each token of the step
        best = rh.rl_sample(z, self.u(T, 1), top_k=torch.full((T,), self.top, dtype=torch.int32, device=dev), capacity=T * self.top, status=st)
        m = best.nnz()
        self.records.append(Recorded(tokens, best.offsets, best.ids[:m], best.support_logq[:m]))

        rel = rh.rl_page_release(plan.kv_lens, v.keep_lens, self.table, self.pool, plan.free_used, page_size=self.page,
                                 n_pages=self.n_pages, held_lens=self.prefix_lens, held_table=self.prefix_table, status=st)
        self.used, self.lens = rel.free_used, v.keep_lens
        at = plan.cu_q[:-1].long() + v.accepted.long()
        self.last[rows] = v.tokens[at[rows]]
        cu, acc, new, lq = plan.cu_q.tolist(), v.accepted.tolist(), v.tokens.tolist(), v.logq.tolist()
        for r in rows.tolist():
            self.texts[r] += new[cu[r]:cu[r] + acc[r] + 1]
            self.logqs[r] += lq[cu[r]:cu[r] + acc[r] + 1]
        return v

    def fork(self):
        """Every live row goes on in the free row after it as well."""
        dev = "cuda"
        parents = torch.tensor([r for r in range(self.R) if self.live[r]], dtype=torch.int32, device=dev)
        children = parents + 1
        f = rh.rl_page_fork(parents, children, self.lens[parents.long()].contiguous(), self.lens, self.table, self.pool, self.used,
                            page_size=self.page, n_pages=self.n_pages, status=self.status)
        rh.rl_page_copy(f.src, f.dst, *self.cache, tokens=f.tokens, status=self.status)
        self.used = f.free_used
        self.last[children.long()] = self.last[parents.long()]
        for r in parents.tolist():
            self.live[r + 1] = True
            self.texts[r + 1], self.logqs[r + 1] = list(self.texts[r]), list(self.logqs[r])

    def compact(self):
        """The live pages together; returns how many there are."""
        c = rh.rl_page_compact(self.lens, self.table, page_size=self.page, n_pages=self.n_pages, prefix_lens=self.prefix_lens,
                               prefix_table=self.prefix_table, status=self.status)
        rh.rl_page_copy(c.src, c.dst, *self.cache, status=self.status)
        self.table, self.prefix_table, self.pool, self.used = c.block_table, c.prefix_table, c.free_pages, c.free_used
        return int(c.free_used.item())


def train_step(drafter: Drafter, records, kind="forward", tail=False, chunk=1024):
    """Loss [N], and gradients of the drafting model's hidden rows and head (token mean), on recorded rows."""
    tokens = torch.cat([r.tokens for r in records])
    offsets = [torch.zeros(1, dtype=torch.int64, device="cuda")]
    for r in records:
        offsets.append(offsets[-1][-1] + r.offsets[1:])
    offsets, ids, logq = torch.cat(offsets), torch.cat([r.ids for r in records]), torch.cat([r.logq for r in records])
    N, H = tokens.numel(), drafter.head.shape[1]
    x = drafter.embed[tokens.long()].contiguous()
    p = rh.DistillParams(kind=kind, tail=tail)
    loss, dX, dW = torch.empty(N, device="cuda"), torch.empty(N, H, device="cuda"), torch.zeros(drafter.head.shape, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for a in range(0, N, chunk):            # a stretch of logits at a time, its gradients in their place
        b = min(a + chunk, N)
        e0, e1 = int(offsets[a]), int(offsets[b])
        z = rh.rl_gemm_bf16_tn(x[a:b], drafter.head, status=status)[0].bfloat16()
        o, d = rh.rl_distill_fwd_bwd(z, offsets[a:b + 1] - e0, ids[e0:e1], logq[e0:e1], torch.full((b - a,), 1.0 / N, device="cuda"), p,
                                     dlogits=z, status=status)
        loss[a:b] = o.loss
        dX[a:b] = rh.rl_gemm_bf16(d, False, drafter.head, True, status=status)[0]
        dW += rh.rl_gemm_bf16(d, True, x[a:b], True, status=status)[0]
    return loss, dX, dW, x, status


def main():
    policy = Policy.random()
    drafter = Drafter.near(policy)
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, 4096, (n,), generator=g).tolist() for n in (37, 16, 150, 5)]
    r = Rollout(policy, drafter, prompts, samples=4, max_new=64)
    taken = []
    for i in range(10):
        v = r.step()
        taken.append(float(v.accepted.sum()) / sum(r.live))
        if i == 4:
            r.fork()
            print("live pages after the fork", r.compact())
    loss, dX, dW, _, status = train_step(drafter, r.records)
    print(f"status {rh.status_names(int(r.status.item()) | int(status.item()))}  drafts accepted a step {sum(taken) / len(taken):.2f} of {r.drafts}  "
          f"tokens {sum(map(len, r.texts))}  distillation loss {float(loss.mean()):.4f}  |dX| {float(dX.norm()):.5f}  |dW| {float(dW.norm()):.5f}")


if __name__ == "__main__":
    main()
