"""The generation operators on representative work: plain torch forms beside the library's calls.

The four operators are the steps of a rollout batch's decode step, in which groups of samples
share one long prompt: page tables and slot maps from request lengths (rl_page_plan), the
step's keys and values into the paged cache (rl_kv_append), attention over a group's shared
prefix and each request's own keys (rl_prefix_attn), and sampling with temperature, top-k,
top-p and min-p from given random numbers, which also writes the sampler support that the
head's loss reads (rl_sample).

`own` false: elementary torch operations.  `own` true: the calls a user's program makes, with
the buffers it keeps from step to step (made on a state's first pass).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ELEM = {"bf16": 2, "fp16": 2, "fp32": 4}
V_HEAD = 151936            # the vocabulary of this repository's head workloads


def listed():
    return [
        # One decode step of 128 sequences in 16 prompt groups: one token each, a new page now and then.
        dict(name="plan_decode", op="plan", R=128, G=16, q_min=1, q_max=1, ctx_max=4096, prefix_max=2048, page=64),
        # First step of a large ragged batch (some requests empty): every token gets its slot.
        dict(name="plan_prompts", op="plan", R=8192, G=1024, q_min=0, q_max=512, ctx_max=0, prefix_max=1000, page=16),
        # The same decode step's keys and values; a few padding tokens.
        dict(name="append_decode", op="append", T=128, Hkv=4, D=128, page=64, dtype="bf16", fused=False),
        # The prompts' keys and values, views of one fused q/k/v projection.
        dict(name="append_prompts", op="append", T=65536, Hkv=8, D=128, page=64, dtype="bf16", fused=True),
        # A handful of samples of a short prompt: latency.
        dict(name="attn_few", op="attn", G=1, per=4, Hq=8, Hkv=2, D=64, page=16, dtype="fp16", q_min=1, q_max=1,
             prefix_min=130, prefix_max=130, own_max=40),
        # A decode step of 128 sequences, 8 samples of each of 16 prompts.
        dict(name="attn_groups", op="attn", G=16, per=8, Hq=16, Hkv=4, D=128, page=64, dtype="bf16", q_min=1, q_max=1,
             prefix_min=300, prefix_max=2048, own_max=512),
        # 64 samples of one long prompt.
        dict(name="attn_long", op="attn", G=1, per=64, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", q_min=1, q_max=1,
             prefix_min=32768, prefix_max=32768, own_max=4096),
        # Requests extended by ragged stretches (a tool's answer, a next turn); some add nothing this step.
        dict(name="attn_extend", op="attn", G=4, per=8, Hq=16, Hkv=2, D=128, page=32, dtype="bf16", q_min=0, q_max=256,
             prefix_min=0, prefix_max=4096, own_max=1024),
        # One row with every knob on: the latency of a single stream.
        dict(name="sample_one", op="sample", N=1, V=V_HEAD, dtype="fp32", K=1, knobs="all"),
        # A decode step of the 128-sequence workload: the label and 16 i.i.d. draws of the whole vocabulary.
        dict(name="sample_draws", op="sample", N=128, V=V_HEAD, dtype="bf16", K=17, knobs="none"),
        # Replayed top-p 0.97 supports, as the replay workloads hold them.
        dict(name="sample_top_p", op="sample", N=256, V=V_HEAD, dtype="fp32", K=1, knobs="top_p"),
        # A large batch of requests that each bring their own settings.
        dict(name="sample_mixed", op="sample", N=1024, V=V_HEAD, dtype="bf16", K=5, knobs="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "sample", "sample"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        R = _log(rng, 1, 8192)
        decode = rng.random() < 0.5
        return dict(op=op, R=R, G=_log(rng, 1, R), q_min=rng.choice([0, 1]), q_max=1 if decode else _log(rng, 2, 512),
                    ctx_max=_log(rng, 1, 4096) if decode else 0, prefix_max=_log(rng, 1, 2048), page=page)
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, T=_log(rng, 1, 65536), Hkv=Hkv, D=rng.choice([64, 128]), page=page,
                    dtype=rng.choice(["bf16", "fp16"]), fused=rng.random() < 0.5)
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        gq = rng.choice([1, 2, 3, 4, 5, 8])
        G = _log(rng, 1, 16)
        per = _log(rng, 1, max(1, 64 // G))
        extend = rng.random() < 0.25
        pre = _log(rng, 1, 32768 // G)
        return dict(op=op, G=G, per=per, Hq=min(Hkv * gq, 32) // Hkv * Hkv, Hkv=Hkv, D=rng.choice([64, 128]),
                    page=page, dtype=rng.choice(["bf16", "fp16"]), q_min=rng.choice([0, 1]),
                    q_max=_log(rng, 2, 128) if extend else 1, prefix_min=rng.choice([0, pre // 2, pre]), prefix_max=pre,
                    own_max=_log(rng, 1, 1024 if extend else 4096))
    return dict(op=op, N=_log(rng, 1, 512), V=rng.choice([1000, 32768, 50257, V_HEAD, _log(rng, 300, V_HEAD)]),
                dtype=rng.choice(["bf16", "fp16", "fp32"]), K=rng.choice([1, 2, 5, 9, 17]),
                knobs=rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]))


# ---- inputs ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _spread(g, lo, hi, n):
    """Lengths spread evenly over [lo, hi], in an order of the seed's: their sum is the case's own."""
    lens = lo + ((torch.arange(n, device="cuda") + 0.5) * (hi - lo + 1) / n).long()
    return lens[torch.randperm(n, generator=g, device="cuda")].to(torch.int32)


def _offsets(lens):
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    return torch.cat([z, torch.cumsum(lens, 0).to(torch.int32)])


def _group_offsets(g, R, G):
    cuts = torch.sort(torch.randint(0, R + 1, (G - 1,), generator=g, device="cuda", dtype=torch.int32)).values
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), cuts,
                      torch.full((1,), R, dtype=torch.int32, device="cuda")])


def _prepare_plan(c, g):
    R, page = c["R"], c["page"]
    q = _spread(g, c["q_min"], c["q_max"], R)
    ctx = _randint(g, 0, c["ctx_max"], R)
    W = -(-(c["ctx_max"] + c["q_max"]) // page)
    had = (ctx.long() + page - 1) // page
    n_pages = R * W + 64
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    used = int(had.sum())
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(W, device="cuda")[None]
    has = cols < had[:, None]
    first = torch.cumsum(had, 0) - had
    table[has] = perm[(first[:, None] + cols)[has]]
    return dict(q_lens=q, ctx_lens=ctx, block_table=table, free_pages=perm,
                free_used=torch.full((1,), used, dtype=torch.int32, device="cuda"), n_pages=n_pages,
                n_tokens=int(q.sum()), group_offsets=_group_offsets(g, R, c["G"]),
                prefix_lens=_randint(g, 0, c["prefix_max"], c["G"]))


def _prepare_append(c, g):
    T, Hkv, D, page, dt = c["T"], c["Hkv"], c["D"], c["page"], DTYPES[c["dtype"]]
    n_pages = -(-T // page) + 8
    slot = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].contiguous()
    slot[torch.rand(T, generator=g, device="cuda") < 0.01] = -1
    if c["fused"]:
        qkv = torch.randn(T, 4 * Hkv, D, generator=g, device="cuda").to(dt)
        k, v = qkv[:, 2 * Hkv:3 * Hkv], qkv[:, 3 * Hkv:]
    else:
        k = torch.randn(T, Hkv, D, generator=g, device="cuda").to(dt)
        v = torch.randn(T, Hkv, D, generator=g, device="cuda").to(dt)
    cache = [torch.zeros(n_pages, Hkv, page, D, dtype=dt, device="cuda") for _ in range(2)]
    return dict(k=k, v=v, slot_map=slot, k_cache=cache[0], v_cache=cache[1])


def _prepare_attn(c, g):
    G, R, page, dt = c["G"], c["G"] * c["per"], c["page"], DTYPES[c["dtype"]]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    q_lens = _spread(g, c["q_min"], c["q_max"], R)
    ctx = _randint(g, 0, max(c["own_max"] - c["q_max"], 0), R)
    kv = ctx + q_lens
    prefix = _randint(g, c["prefix_min"], c["prefix_max"], G)
    W, WP = -(-max(c["own_max"], c["q_max"]) // page), max(1, -(-c["prefix_max"] // page))
    n_pages = R * W + G * WP + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    T = int(q_lens.sum())
    kc, vc = [torch.empty(n_pages, Hkv, page, D, dtype=dt, device="cuda") for _ in range(2)]
    step = max(1, (1 << 27) // (Hkv * page * D))
    for a in range(0, n_pages, step):
        b = min(n_pages, a + step)
        kc[a:b] = torch.randn(b - a, Hkv, page, D, generator=g, device="cuda").to(dt)
        vc[a:b] = torch.randn(b - a, Hkv, page, D, generator=g, device="cuda").to(dt)
    # queries a little longer than the keys, so that some keys stand out as trained heads' do
    q = (1.5 * torch.randn(T, Hq, D, generator=g, device="cuda")).to(dt)
    return dict(q=q, k_cache=kc, v_cache=vc, cu_q=_offsets(q_lens), kv_lens=kv,
                block_table=perm[:R * W].view(R, W).contiguous(),
                group_offsets=torch.arange(G + 1, device="cuda", dtype=torch.int32) * c["per"],
                prefix_lens=prefix, prefix_table=perm[R * W:R * W + G * WP].view(G, WP).contiguous(),
                max_q=c["q_max"], max_kv=max(c["own_max"], c["q_max"]), max_prefix=c["prefix_max"],
                scale=1.0 / math.sqrt(D))


def _prepare_sample(c, g):
    N, V, K, kn = c["N"], c["V"], c["K"], c["knobs"]
    # a broad bulk with a heavy upper tail of each row's own width, and a few likely tokens
    z = torch.randn(N, V, generator=g, device="cuda")
    z = z * (1.5 + 1.5 * torch.rand(N, 1, generator=g, device="cuda"))
    at = torch.randint(0, V, (N, 24), generator=g, device="cuda")
    z.scatter_(1, at, 8 + 6 * torch.rand(N, 24, generator=g, device="cuda"))
    # the padding rows of the vocabulary, and a grammar's mask in some rows
    z[:, V - V // 500:] = float("-inf")
    masked = (torch.rand(N, generator=g, device="cuda") < 0.1)[:, None] & (torch.arange(V, device="cuda") % 3 != 0)[None]
    z = z.masked_fill_(masked, float("-inf")).to(DTYPES[c["dtype"]])
    u = (torch.randint(0, 1 << 24, (N, K), generator=g, device="cuda").float() + 0.5) / (1 << 24)
    u.clamp_(max=1 - 2.0 ** -24)
    rnd = lambda: torch.rand(N, generator=g, device="cuda")  # noqa: E731
    temp = 0.6 + 0.6 * rnd() if kn in ("all", "mixed") else None
    top_k = torch.randint(5, min(V, 400), (N,), generator=g, device="cuda", dtype=torch.int32) \
        if kn in ("top_k", "all", "mixed") else None
    top_p = 0.97 * torch.ones(N, device="cuda") if kn == "top_p" else 0.8 + 0.19 * rnd() if kn in ("all", "mixed") else None
    min_p = 0.01 + 0.1 * rnd() if kn in ("min_p", "all", "mixed") else None
    if kn == "mixed":       # each row with its own choice of knobs; some with none
        pick = torch.randint(0, 8, (N,), generator=g, device="cuda")
        top_k[pick % 2 == 0] = 0
        top_p[(pick // 2) % 2 == 0] = 1.0
        min_p[pick // 4 == 0] = 0.0
        temp[pick == 5] = 0.0                # greedy
    # room for every row's support: no row keeps more than a stretch of the vocabulary here
    cap = N * (max(K, 400) if kn in ("none", "top_k", "all", "min_p") else min(V, 16384))
    return dict(logits=z, u=u, temperature=temp, top_k=top_k, top_p=top_p, min_p=min_p, cap=cap)


def prepare(case, seed):
    g = _gen(seed)
    s = {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn, "sample": _prepare_sample}[case["op"]](case, g)
    s["op"], s["page"], s["keep"] = case["op"], case["page"] if "page" in case else 0, {}
    return s


# ---- plain forms ----------------------------------------------------------------------

def _plain_plan(s):
    page, n_free, table = s["page"], s["free_pages"].numel(), s["block_table"].clone()
    q, ctx = s["q_lens"].long(), s["ctx_lens"].long()
    R, W, T = q.numel(), table.shape[1], s["n_tokens"]
    had, need = (ctx + page - 1) // page, (ctx + q + page - 1) // page
    new = need - had
    first = torch.cumsum(new, 0) - new
    cols = torch.arange(W, device=q.device)[None]
    takes = (cols >= had[:, None]) & (cols < need[:, None])
    pool = s["free_used"].long() + first[:, None] + cols - had[:, None]
    table = torch.where(takes, s["free_pages"][pool.clamp(0, n_free - 1)], table)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=q.device), torch.cumsum(q, 0)])
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu, t, right=True) - 1
    at = ctx[r] + t - cu[r]
    slot = table[r, at // page].long() * page + at % page
    g = torch.searchsorted(s["group_offsets"].long(), r, right=True) - 1
    return dict(cu_q=cu.to(torch.int32), kv_lens=(ctx + q).to(torch.int32), slot_map=slot,
                positions=(s["prefix_lens"][g] + at).to(torch.int32), block_table=table,
                free_used=(s["free_used"] + new.sum()).to(torch.int32))


def _plain_append(s):
    page, Hkv, D = s["page"], s["k"].shape[1], s["k"].shape[2]
    slot = s["slot_map"]
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    ok = slot >= 0
    sl = slot[ok]
    kc[sl // page, :, sl % page] = s["k"][ok]
    vc[sl // page, :, sl % page] = s["v"][ok]
    return dict(k_cache=kc, v_cache=vc)


def _part(scores, seen, v, eq):
    """(max, sum, numerator) of one part of the keys; `scores` [..., keys], unseen keys out."""
    scores = scores.masked_fill(~seen, float("-inf"))
    m = scores.amax(-1)
    e = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m)[..., None])
    return m, e.sum(-1), torch.einsum(eq, e, v)


def _plain_attn(s):
    q, kc, vc, page = s["q"], s["k_cache"], s["v_cache"], s["page"]
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    x = Hq // Hkv
    dev = q.device
    cu, kv, go = s["cu_q"].long(), s["kv_lens"].long(), s["group_offsets"].long()
    R, G = kv.numel(), go.numel() - 1
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[r]
    g = torch.searchsorted(go, r, right=True) - 1
    qf = (q.float() * s["scale"]).view(T, Hkv, x, D)

    def pages(cache, table):        # [rows, Hkv, keys, D]
        return cache[table.long()].float().permute(0, 2, 1, 3, 4).reshape(table.shape[0], Hkv, -1, D)

    # the group's prefix, once for the queries of the group
    Tg = cu[go]
    j = t - Tg[g]
    Mg = max(1, s["max_q"] * -(-R // G))
    qp = torch.zeros(G, Mg, Hkv, x, D, device=dev)
    qp[g, j] = qf
    kp, vp = pages(kc, s["prefix_table"]), pages(vc, s["prefix_table"])
    seen = torch.arange(kp.shape[2], device=dev) < s["prefix_lens"].long()[:, None, None, None, None]
    m1, l1, o1 = _part(torch.einsum("gmhxd,ghkd->ghxmk", qp, kp), seen, vp, "ghxmk,ghkd->gmhxd")
    m1, l1, o1 = m1.permute(0, 3, 1, 2)[g, j], l1.permute(0, 3, 1, 2)[g, j], o1[g, j]
    # each request's own keys, causal within the step
    qo = torch.zeros(R, s["max_q"], Hkv, x, D, device=dev)
    qo[r, i] = qf
    ko, vo = pages(kc, s["block_table"]), pages(vc, s["block_table"])
    last = kv[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(s["max_q"], device=dev)
    seen = torch.arange(ko.shape[2], device=dev) <= torch.minimum(last, kv[:, None] - 1)[:, None, None, :, None]
    m2, l2, o2 = _part(torch.einsum("rqhxd,rhkd->rhxqk", qo, ko), seen, vo, "rhxqk,rhkd->rqhxd")
    m2, l2, o2 = m2.permute(0, 3, 1, 2)[r, i], l2.permute(0, 3, 1, 2)[r, i], o2[r, i]
    m = torch.maximum(m1, m2)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    a1, a2 = torch.exp(m1 - m0), torch.exp(m2 - m0)
    den = a1 * l1 + a2 * l2
    o = (a1[..., None] * o1 + a2[..., None] * o2) / torch.where(den > 0, den, torch.ones_like(den))[..., None]
    return dict(out=o.reshape(T, Hq, D).to(q.dtype), lse=(m0 + torch.log(den)).reshape(T, Hq))


def _row(v, N, default, dev):
    return torch.full((N, 1), float(default), dtype=torch.float64, device=dev) if v is None else v.double()[:, None]


def _plain_sample(s):
    z = s["logits"].double()                     # borders of sets and sums: 64 bits
    N, V = z.shape
    K, cap, dev = s["u"].shape[1], s["cap"], z.device
    T, p, mp, k = (_row(s[n], N, d, dev) for n, d in (("temperature", 1), ("top_p", 1), ("min_p", 0), ("top_k", 0)))
    greedy = T == 0
    k = torch.where(greedy, torch.ones_like(k), torch.where((k <= 0) | (k > V), torch.full_like(k, V), k))
    zmax = z.amax(1, keepdim=True)
    x = (z - zmax) / torch.where(greedy, torch.ones_like(T), T)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    w = torch.exp(x)
    ws = w.gather(1, order)
    keep = (torch.arange(V, device=dev)[None] < k) & (ws >= mp.clamp(min=2.0 ** -100, max=1))
    ws = ws * keep
    cum = torch.cumsum(ws, 1)
    keep &= (cum - ws < p * cum[:, -1:]) | (p >= 1)
    S = torch.zeros(N, V, dtype=torch.bool, device=dev).scatter_(1, order, keep)
    del order, ws, cum, keep
    w = w * S
    cdf = torch.cumsum(w, 1)
    total = cdf[:, -1:]
    tok = torch.searchsorted(cdf, s["u"].double() * total, right=True).clamp_(max=V - 1)
    lq = torch.where(greedy, torch.zeros_like(x), x - torch.log(total))
    del cdf, w
    logq = lq.gather(1, tok)
    replayed = ((k < V) | (p < 1) | (mp > 0)).view(N)
    # the support: the kept set of a truncated row, the other draws (ascending) of a whole one
    count = torch.where(replayed, S.sum(1), torch.full((N,), K - 1, device=dev))
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(count, 0)])
    S &= replayed[:, None]
    place = torch.cumsum(S, 1) - 1 + off[:-1, None]
    place = torch.where(S, place.clamp(max=cap), torch.full_like(place, cap)).view(-1)
    ids = torch.zeros(cap + 1, dtype=torch.int32, device=dev)
    slq = torch.zeros(cap + 1, dtype=torch.float32, device=dev)
    ids.scatter_(0, place, torch.arange(V, device=dev, dtype=torch.int32).repeat(N))
    slq.scatter_(0, place, lq.float().view(-1))
    if K > 1:
        d = torch.sort(tok[:, 1:], dim=1).values
        at = off[:-1, None] + torch.arange(K - 1, device=dev)
        at = torch.where(replayed[:, None], torch.full_like(at, cap), at.clamp(max=cap))
        ids.scatter_(0, at.view(-1), d.to(torch.int32).view(-1))
        slq.scatter_(0, at.view(-1), lq.gather(1, d).float().view(-1))
    return dict(tokens=tok.to(torch.int32), logq=logq.float(), offsets=off, ids=ids[:cap], support_logq=slq[:cap],
                replayed=replayed.to(torch.uint8))


# ---- the library's calls ---------------------------------------------------------------

def _own_plan(s):
    import lm_head_gb300 as rh
    k = s["keep"]
    p = rh.rl_page_plan(s["q_lens"], s["ctx_lens"], s["block_table"], s["free_pages"], page_size=s["page"],
                        n_pages=s["n_pages"], n_tokens=s["n_tokens"], free_used=s["free_used"],
                        group_offsets=s["group_offsets"], prefix_lens=s["prefix_lens"], out=k.get("plan"))
    k["plan"] = p
    return dict(cu_q=p.cu_q, kv_lens=p.kv_lens, slot_map=p.slot_map, positions=p.positions,
                block_table=s["block_table"], free_used=p.free_used)


def _own_append(s):
    import lm_head_gb300 as rh
    s["keep"]["status"] = rh.rl_kv_append(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"],
                                          status=s["keep"].get("status"))
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_attn(s):
    import lm_head_gb300 as rh
    a = rh.rl_prefix_attn(s["q"], s["k_cache"], s["v_cache"], s["cu_q"], s["kv_lens"], s["block_table"],
                          max_q=s["max_q"], max_kv=s["max_kv"], group_offsets=s["group_offsets"],
                          prefix_lens=s["prefix_lens"], prefix_table=s["prefix_table"], max_prefix=s["max_prefix"],
                          scale=s["scale"], out=s["keep"].get("attn"))
    s["keep"]["attn"] = a
    return dict(out=a.out, lse=a.lse)


def _own_sample(s):
    import lm_head_gb300 as rh
    o = rh.rl_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], capacity=s["cap"], out=s["keep"].get("sample"))
    s["keep"]["sample"] = o
    return dict(tokens=o.tokens, logq=o.logq, offsets=o.offsets, ids=o.ids, support_logq=o.support_logq,
                replayed=o.replayed)


def run(state):
    forms = (_own_plan, _own_append, _own_attn, _own_sample) if own else (_plain_plan, _plain_append, _plain_attn, _plain_sample)
    return forms[("plan", "append", "attn", "sample").index(state["op"])](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "plan":
        T = c["R"] * (c["q_min"] + c["q_max"]) / 2
        new = T / c["page"] + (c["R"] / 2 if c["ctx_max"] == 0 else 0)
        return {"bytes": 8 * c["R"] + 8 * (c["R"] + 1) + 12 * T + 8 * new + 8 * c["G"], "flops": 0}
    if c["op"] == "append":
        return {"bytes": c["T"] * (8 + 4 * c["Hkv"] * c["D"] * ELEM[c["dtype"]]), "flops": 0}
    if c["op"] == "attn":
        R = c["G"] * c["per"]
        q = (c["q_min"] + c["q_max"]) / 2
        pre, kv = (c["prefix_min"] + c["prefix_max"]) / 2, max(c["own_max"] - c["q_max"], 0) / 2 + q
        T = R * q
        e = ELEM[c["dtype"]]
        return {"bytes": 2 * (c["G"] * pre + R * kv) * c["Hkv"] * c["D"] * e + T * c["Hq"] * (2 * c["D"] * e + 4),
                "flops": 4 * c["Hq"] * c["D"] * T * (pre + kv - max(q - 1, 0) / 2)}
    # every logit once; where a total over the vocabulary is taken, one exponential and one sum of each
    return {"bytes": c["N"] * c["V"] * ELEM[c["dtype"]] + 12 * c["N"] * c["K"], "flops": 2 * c["N"] * c["V"]}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_attn(s):
    q, page = s["q"].double(), s["page"]
    T, Hq, D = q.shape
    Hkv = s["k_cache"].shape[1]
    cu, kv, go, pl = (s[n].tolist() for n in ("cu_q", "kv_lens", "group_offsets", "prefix_lens"))
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    group = np.searchsorted(np.asarray(go), np.arange(len(kv)), side="right") - 1
    heads = torch.arange(Hq, device="cuda") // (Hq // Hkv)

    def keys(cache, table, n):      # [Hkv, n, D]
        return cache[table[:-(-n // page)].long()].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n].double()

    for r in range(len(kv)):
        n, P, L = cu[r + 1] - cu[r], pl[group[r]], kv[r]
        if n == 0 or P + L == 0:
            continue
        k, v = (torch.cat([keys(s[c], s["prefix_table"][group[r]], P), keys(s[c], s["block_table"][r], L)], 1)[heads]
                for c in ("k_cache", "v_cache"))
        a = torch.bmm(q[cu[r]:cu[r + 1]].transpose(0, 1), k.transpose(1, 2)) * s["scale"]
        limit = P + L - n + torch.arange(n, device="cuda")
        a = a.masked_fill(torch.arange(P + L, device="cuda")[None] > limit[:, None], float("-inf"))
        lse[cu[r]:cu[r + 1]] = torch.logsumexp(a, 2).T
        out[cu[r]:cu[r + 1]] = torch.bmm(torch.softmax(a, 2), v).transpose(0, 1)
    return dict(out=out, lse=lse)


def _exact_sample(s):
    """The definition row by row: the kept set by ranks, then the cumulative sums over it."""
    z = s["logits"].cpu().double().numpy()
    N, V = z.shape
    u, K, cap = s["u"].cpu().double().numpy(), s["u"].shape[1], s["cap"]
    knob = {n: None if s[n] is None else s[n].cpu().double().numpy() for n in ("temperature", "top_k", "top_p", "min_p")}
    at = lambda n, r, d: d if knob[n] is None else float(knob[n][r])  # noqa: E731
    tok, logq = np.zeros((N, K), np.int32), np.zeros((N, K))
    off, ids, slq, rep = [0], np.zeros(cap, np.int32), np.zeros(cap), np.zeros(N, np.uint8)
    for r in range(N):
        T, k, p, mp = at("temperature", r, 1), int(at("top_k", r, 0)), at("top_p", r, 1), at("min_p", r, 0)
        k = 1 if T == 0 else k if 0 < k <= V else V
        x = (z[r] - z[r].max()) / (T or 1.0)
        cand = np.flatnonzero(x >= math.log(min(max(mp, 2.0 ** -100), 1.0)))
        if k < V or p < 1:
            cand = cand[np.argsort(-x[cand], kind="stable")][:k]
        if p < 1:
            c = np.cumsum(np.exp(x[cand]))
            cand = cand[:1 + int(np.count_nonzero(c[:-1] < p * c[-1]))]
        cand = np.sort(cand)
        c = np.cumsum(np.exp(x[cand]))
        lq = x[cand] - math.log(c[-1]) if T else np.zeros(1)
        d = np.minimum(np.searchsorted(c, u[r] * c[-1], side="right"), len(cand) - 1)
        tok[r], logq[r] = cand[d], lq[d]
        rep[r] = k < V or p < 1 or mp > 0
        keep = np.arange(len(cand)) if rep[r] else np.sort(d[1:])
        a, b = off[-1], off[-1] + len(keep)
        n = max(0, min(b, cap) - a)
        ids[a:a + n], slq[a:a + n] = cand[keep][:n], lq[keep][:n]
        off.append(b)
    return dict(tokens=tok, logq=logq, offsets=np.asarray(off, np.int64), ids=ids, support_logq=slq, replayed=rep)


def exact(case, seed):
    c = case
    if c["op"] == "attn" and work(c)["flops"] < 1e12:
        return _exact_attn(prepare(case, seed))
    if c["op"] == "sample" and c["N"] * c["V"] <= 60_000_000:
        return _exact_sample(prepare(case, seed))
    return None             # page plans and cache writes compute no numbers of their own
