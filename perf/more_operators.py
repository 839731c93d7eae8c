"""Operators of speculative rollouts on representative work: plain torch forms beside the library's calls.

A rollout engine lets a small model draft several tokens of each request, runs the target on
them in one step and keeps what the target's own sampling would have given (rl_verify).  The
pages of what it turned down go back to the pool (rl_page_release); a sequence that is
continued in several ways is forked, sharing its full pages and copying the last one
(rl_page_fork, rl_page_copy); before the trainer takes the memory over, the live pages are moved
together (rl_page_compact, rl_page_copy).  The drafting model is then trained on the target's
top tokens, which the rollout recorded as support rows (rl_distill_fwd_bwd).

`own` false: elementary torch operations.  `own` true: the calls a user's program makes, with
the buffers it keeps from step to step (made on a state's first pass).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ELEM = {"bf16": 2, "fp16": 2, "fp32": 4}
V_HEAD = 151936            # the vocabulary of this repository's head workloads
NEG = float("-inf")


def listed():
    return [
        # One stream with four drafted tokens, each model's own temperature: latency.
        dict(name="verify_one", op="verify", R=1, q_min=5, q_max=5, V=V_HEAD, dtype="fp32", target="dense", draft="dense",
             temp=True),
        # The 128-sequence workload's step with four drafts each, whole distributions on both sides.
        dict(name="verify_batch", op="verify", R=128, q_min=5, q_max=5, V=V_HEAD, dtype="bf16", target="dense", draft="dense",
             temp=False),
        # Requests with their own settings: truncated targets as support rows beside whole ones, drafts
        # sampled from truncated rows, none to eight of them.
        dict(name="verify_mixed", op="verify", R=256, q_min=1, q_max=9, V=V_HEAD, dtype="bf16", target="mixed", draft="rows",
             temp=True),
        # After a verified step of 128 requests: a page back now and then.
        dict(name="release_step", op="release", R=128, len_max=4096, drop=8, page=64, shared=0.25),
        # The end of a large batch: half the requests are done and give all they have back.
        dict(name="release_done", op="release", R=8192, len_max=1024, drop=-1, page=16, shared=0.25),
        # A few continuations of a sequence, a small model's cache.
        dict(name="fork_few", op="fork", R=16, C=4, len_max=300, page=16, Hkv=2, D=64, L=4, dtype="fp16"),
        # Every request of a batch branched into four, the last pages copied in eight layers.
        dict(name="fork_batch", op="fork", R=1024, C=768, len_max=1024, page=64, Hkv=8, D=128, L=8, dtype="bf16"),
        # A small pool, mostly tables and lists.
        dict(name="compact_small", op="compact", R=32, G=4, len_max=512, page=16, Hkv=2, D=64, L=2, dtype="bf16", spread=2.0),
        # A large cache at the end of a rollout, one page in two live and spread over it.
        dict(name="compact_large", op="compact", R=512, G=32, len_max=2048, page=64, Hkv=4, D=128, L=4, dtype="bf16",
             spread=2.0),
        # A drafting head of a small vocabulary on one request's tokens.
        dict(name="distill_small", op="distill", N=64, V=32768, dtype="fp32", k_min=20, k_max=20, kind="forward", tail=True,
             T=1.0),
        # A batch of tokens against up to 64 recorded top tokens each; some rows recorded none.
        dict(name="distill_top", op="distill", N=4096, V=V_HEAD, dtype="bf16", k_min=0, k_max=64, kind="forward", tail=False,
             T=1.0),
        # The other direction in fp32 logits, with the rest of the vocabulary as one outcome.
        dict(name="distill_tail", op="distill", N=2048, V=V_HEAD, dtype="fp32", k_min=1, k_max=128, kind="reverse", tail=True,
             T=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "release", "fork", "compact", "distill", "distill"])
    page = rng.choice([16, 32, 64, 128])
    if op in ("verify", "distill"):
        V = rng.choice([1000, 32768, 50257, V_HEAD, _log(rng, 300, V_HEAD)])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "verify":
        R = _log(rng, 1, 256)
        q_max = _log(rng, 1, 12)
        most = int(1.2e8 if dtype != "fp32" else 6e7)
        while R * q_max * V > most:
            R = max(1, R // 2)
        return dict(op=op, R=R, q_min=rng.randint(0, q_max), q_max=q_max, V=V, dtype=dtype,
                    target=rng.choice(["dense", "rows", "mixed"]), draft=rng.choice(["dense", "rows", "mixed", "sure"]),
                    temp=rng.random() < 0.5)
    if op == "release":
        return dict(op=op, R=_log(rng, 1, 8192), len_max=_log(rng, 1, 1024 if page < 64 else 4096),
                    drop=rng.choice([-1, 1, 8, 64]), page=page, shared=rng.choice([0.0, 0.25, 0.9]))
    if op in ("fork", "compact"):
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        R = _log(rng, 2, 512)
        # the cache at most that of the largest listed case
        tokens = int(2.0e9 / (Hkv * D))
        L = _log(rng, 1, 8)
        len_max = max(1, min(_log(rng, 1, 2048), tokens // (R * L) - page))
        c = dict(op=op, R=R, len_max=len_max, page=page, Hkv=Hkv, D=D, L=L, dtype=rng.choice(["bf16", "fp16"]))
        if op == "fork":
            return dict(c, C=_log(rng, 1, max(1, R - 1)))
        return dict(c, G=_log(rng, 1, 32), spread=rng.choice([1.0, 1.3, 2.0]))
    N = min(_log(rng, 1, 4096), int((6e8 if dtype != "fp32" else 3e8) / V))
    kind = rng.choice(["forward", "reverse", "jsd"])
    k_max = _log(rng, 1, min(256, V // 4))
    return dict(op=op, N=N, V=V, dtype=dtype, k_min=rng.choice([0, 1, k_max]), k_max=k_max, kind=kind,
                tail=kind != "forward" or rng.random() < 0.5, T=rng.choice([0.7, 1.0, 2.0]))


# ---- inputs ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _rand(g, *n):
    return torch.rand(*n, generator=g, device="cuda")


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _spread(g, lo, hi, n):
    """Lengths spread evenly over [lo, hi], in an order of the seed's: their sum is the case's own."""
    lens = lo + ((torch.arange(n, device="cuda") + 0.5) * (hi - lo + 1) / n).long()
    return lens[torch.randperm(n, generator=g, device="cuda")].to(torch.int32)


def _offsets(lens, dtype=torch.int32):
    return torch.cat([torch.zeros(1, dtype=dtype, device="cuda"), torch.cumsum(lens, 0).to(dtype)])


def _uniform(g, *n):
    u = (torch.randint(0, 1 << 24, n, generator=g, device="cuda").float() + 0.5) / (1 << 24)
    return u.clamp_(max=1 - 2.0 ** -24)


def _logits(g, N, V):
    """A broad bulk with an upper tail of each row's own width, and a few likely tokens."""
    z = torch.randn(N, V, generator=g, device="cuda")
    z *= 1.5 + 1.5 * _rand(g, N, 1)
    for _ in range(12):     # (one place a row at a time: no two values meet)
        at = torch.randint(0, V, (N, 1), generator=g, device="cuda")
        z.scatter_(1, at, 8 + 6 * _rand(g, N, 1))
    return z


def _support(z, T, g, most, mass):
    """Truncated rows as a sampler records them: ids ascending, log-probabilities renormalised."""
    N, V = z.shape
    top, ids = torch.topk(z.float() / T[:, None].clamp(min=1e-3), min(most, V), dim=1)
    p = torch.softmax(top.double(), 1)
    keep = torch.cumsum(p, 1) - p < mass
    keep &= torch.arange(p.shape[1], device="cuda")[None] < torch.where(T > 0, 1 << 30, 1)[:, None]
    p = torch.where(keep, p, torch.zeros_like(p))
    logq = torch.log(p / p.sum(1, keepdim=True)).float()
    order = torch.sort(torch.where(keep, ids, V), dim=1).indices
    ids, logq, keep = ids.gather(1, order), logq.gather(1, order), keep.gather(1, order)
    return dict(offsets=_offsets(keep.sum(1), torch.int64), ids=ids[keep].to(torch.int32), logq=logq[keep].contiguous())


def _dist(z, T, form, g, temp):
    """What the program holds of the rows' distributions: logits, support rows, or each row one of them."""
    d = dict(logits=None, temperature=None, offsets=None, ids=None, logq=None, replayed=None)
    N = z.shape[0]
    if form != "rows":
        d["logits"], d["temperature"] = z, T if temp else None
    if form != "dense":
        d.update(_support(z, T, g, 512, 0.97))
        d["replayed"] = torch.ones(N, dtype=torch.uint8, device="cuda") if form == "rows" else \
            (_rand(g, N) < 0.5).to(torch.uint8)
    return d


def _prepare_verify(c, g):
    R, V, dt = c["R"], c["V"], DTYPES[c["dtype"]]
    q = _spread(g, c["q_min"], c["q_max"], R)
    cu, T = _offsets(q), int(q.sum())
    n = max(T, 1)
    z = _logits(g, n, V)
    # the drafting model: the target's logits less sharp, and its own error
    zd = (0.9 * z + 0.7 * torch.randn(n, V, generator=g, device="cuda")).to(dt)
    z[:, V - V // 500:] = NEG           # the padding rows of the vocabulary
    z = z.to(dt)
    if c["temp"]:       # a request's own; some are greedy
        temp = (0.6 + 0.6 * _rand(g, n)) * (_rand(g, n) > 0.1)
    else:
        temp = torch.ones(n, device="cuda")
    target = _dist(z, temp, c["target"], g, c["temp"])
    if c["draft"] == "sure":
        draft = None
        likely = torch.argmax(zd, 1)
        tok = torch.where(_rand(g, n) < 0.8, likely, torch.randint(0, V, (n,), generator=g, device="cuda"))
    else:
        draft = _dist(zd, torch.ones(n, device="cuda"), c["draft"], g, False)
        p = torch.softmax(zd.float(), 1)
        if c["draft"] != "dense":       # drafted from the rows that are held
            rows = torch.repeat_interleave(torch.arange(n, device="cuda"), draft["offsets"].diff())
            held = torch.zeros_like(p)
            held[rows, draft["ids"].long()] = torch.exp(draft["logq"])
            p = torch.where(draft["replayed"].bool()[:, None], held, p)
        tok = torch.multinomial(p, 1, generator=g)[:, 0]
    step = torch.randint(0, V, (n + 1,), generator=g, device="cuda", dtype=torch.int32)
    step[1:] = tok.to(torch.int32)      # row t's candidate is the token after it
    return dict(step_tokens=step[:T].contiguous(), cu_q=cu, u=_uniform(g, n)[:T].contiguous(), u_next=_uniform(g, R),
                target=target, draft=draft, V=V, ctx_lens=_randint(g, 0, 4096, R), T=T)


def _tables(g, R, W, lens, page, shared):
    """Page tables of requests, some of which share their first pages with the request before them; the pages
    lie in the order of handing out.  Returns the table, the pool's order, how many were handed out."""
    had = (lens.long() + page - 1) // page
    cols = torch.arange(W, device="cuda")[None]
    follows = (_rand(g, R) < shared) & (torch.arange(R, device="cuda") % 2 == 1)
    before = torch.minimum(torch.roll(lens.long(), 1) // page, lens.long() // page)
    n_shared = torch.where(follows, (before * _rand(g, R)).long(), torch.zeros_like(before))
    takes = (cols < had[:, None]) & (cols >= n_shared[:, None])
    n_pages = R * W + 64
    pool = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    place = torch.cumsum(takes.view(-1), 0).view(R, W) - 1
    table[takes] = pool[place[takes]]
    table = torch.where(cols < n_shared[:, None], torch.roll(table, 1, 0), table).contiguous()
    return table, pool, int(takes.sum()), n_pages


def _prepare_release(c, g):
    R, page = c["R"], c["page"]
    W = -(-c["len_max"] // page)
    lens = _spread(g, 1, c["len_max"], R)
    table, pool, used, n_pages = _tables(g, R, W, lens, page, c["shared"])
    if c["drop"] < 0:
        keep = torch.where(_rand(g, R) < 0.5, lens, torch.zeros_like(lens))
    else:
        keep = (lens - _randint(g, 0, c["drop"], R)).clamp(min=0)
    return dict(kv_lens=lens, keep_lens=keep, block_table=table, free_pages=pool,
                free_used=torch.full((1,), used, dtype=torch.int32, device="cuda"), n_pages=n_pages)


def _caches(g, L, n_pages, Hkv, page, D, dt):
    kc, vc = [torch.empty(L, n_pages, Hkv, page, D, dtype=dt, device="cuda") for _ in range(2)]
    step = max(1, (1 << 27) // (Hkv * page * D))
    for x in (kc, vc):
        for layer in range(L):
            for a in range(0, n_pages, step):
                b = min(n_pages, a + step)
                x[layer, a:b] = torch.randn(b - a, Hkv, page, D, generator=g, device="cuda").to(dt)
    return kc, vc


def _prepare_fork(c, g):
    R, C, page = c["R"], c["C"], c["page"]
    P = R - C                           # the rows that there are; the others are free
    W = -(-c["len_max"] // page)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    lens[:P] = _spread(g, 1, c["len_max"], P)
    rows = torch.randperm(R, generator=g, device="cuda")
    lens = lens[torch.argsort(rows)].contiguous()               # row rows[i] has the i-th length
    children = rows[P:].to(torch.int32)
    parents = rows[torch.arange(C, device="cuda") % P].to(torch.int32)
    at = lens[parents.long()]
    # most go on from the parent's end, some from an earlier token
    back = (at.float() * _rand(g, C)).to(torch.int32)
    fork = torch.where(_rand(g, C) < 0.75, at, back)
    had = (lens.long() + page - 1) // page
    n_pages = P * W + C + 16
    pool = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    has = torch.arange(W, device="cuda")[None] < had[:, None]
    table[has] = pool[:int(has.sum())]
    kc, vc = _caches(g, c["L"], n_pages, c["Hkv"], page, c["D"], DTYPES[c["dtype"]])
    return dict(parents=parents, children=children, lens=fork.to(torch.int32), kv_lens=lens, block_table=table, free_pages=pool,
                free_used=torch.full((1,), int(has.sum()), dtype=torch.int32, device="cuda"), n_pages=n_pages,
                k_cache=kc, v_cache=vc)


def _prepare_compact(c, g):
    R, G, page = c["R"], c["G"], c["page"]
    W = -(-c["len_max"] // page)
    lens = _spread(g, 0, c["len_max"], R + G)
    table, pool, _, _ = _tables(g, R + G, W, lens, page, 0.25)
    # the pages in use lie anywhere in a cache `spread` times what they would be unshared
    n_pages = int(int(((lens.long() + page - 1) // page).sum()) * c["spread"]) + 1
    where = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    inv = torch.empty_like(pool)
    inv[pool.long()] = torch.arange(pool.numel(), device="cuda", dtype=torch.int32)
    table = torch.where(table >= 0, where[inv[table.long().clamp(min=0)].long().clamp(max=n_pages - 1)], table)
    kc, vc = _caches(g, c["L"], n_pages, c["Hkv"], page, c["D"], DTYPES[c["dtype"]])
    return dict(kv_lens=lens[:R].contiguous(), block_table=table[:R].contiguous(), prefix_lens=lens[R:].contiguous(),
                prefix_table=table[R:].contiguous(), n_pages=n_pages, k_cache=kc, v_cache=vc)


def _prepare_distill(c, g):
    N, V, T = c["N"], c["V"], c["T"]
    z = _logits(g, N, V)
    teacher = 1.1 * z + 0.5 * torch.randn(N, V, generator=g, device="cuda")
    z = z.to(DTYPES[c["dtype"]])
    logq = torch.log_softmax(teacher / T, 1) if c["tail"] else teacher      # top logits will do where they are renormalised
    k = _spread(g, c["k_min"], c["k_max"], N)
    top, ids = torch.topk(logq, c["k_max"], dim=1)
    keep = torch.arange(c["k_max"], device="cuda")[None] < k[:, None]
    order = torch.sort(torch.where(keep, ids, V), dim=1).indices
    top, ids, keep = top.gather(1, order), ids.gather(1, order), keep.gather(1, order)
    dloss = torch.where(_rand(g, N) < 0.1, torch.zeros(N, device="cuda"), 0.5 + _rand(g, N)) / N     # some prompt tokens
    if c["dtype"] == "fp16":
        dloss = dloss * 65536           # scaled as training in fp16 does it
    return dict(logits=z, offsets=_offsets(k, torch.int64), ids=ids[keep].to(torch.int32), logq=top[keep].contiguous(),
                dloss=dloss, kind=c["kind"], tail=c["tail"], T=T, beta=0.3)


PREPARE = {"verify": _prepare_verify, "release": _prepare_release, "fork": _prepare_fork, "compact": _prepare_compact,
           "distill": _prepare_distill}


def prepare(case, seed):
    s = PREPARE[case["op"]](case, _gen(seed))
    s["op"], s["page"], s["keep"] = case["op"], case.get("page", 0), {}
    return s


# ---- plain forms ----------------------------------------------------------------------
# Borders of sums and sets are decided in 64 bits.

def _log_total(z, temp):
    """Row maximum, its first place, and the log of the sum of exp((z - max) / T); rows of T = 0: the place alone."""
    zm, at = z.max(1)
    return zm, at, torch.log(torch.exp((z - zm[:, None]) / torch.where(temp > 0, temp, torch.ones_like(temp))[:, None]).sum(1))


def _temps(d, n, dev):
    return torch.ones(n, dtype=torch.float64, device=dev) if d["temperature"] is None else d["temperature"].double()


def _log_prob(d, x, V):
    """log of each row's probability of its token x, in 64 bits; -inf where it has none."""
    n, dev = x.numel(), x.device
    out = torch.full((n,), NEG, dtype=torch.float64, device=dev)
    if d["logits"] is not None:
        z, T = d["logits"][:n].double(), _temps(d, d["logits"].shape[0], dev)[:n]
        zm, at, lt = _log_total(z, T)
        lp = (z.gather(1, x[:, None])[:, 0] - zm) / torch.where(T > 0, T, torch.ones_like(T)) - lt
        out = torch.where(T > 0, lp, torch.where(at == x, torch.zeros_like(lp), torch.full_like(lp, NEG)))
    if d["offsets"] is not None:
        rows = torch.searchsorted(d["offsets"], torch.arange(d["ids"].numel(), device=dev), right=True) - 1
        keys = rows * V + d["ids"]
        want = torch.arange(n, device=dev) * V + x
        i = torch.searchsorted(keys, want).clamp(max=max(keys.numel() - 1, 0))
        found = torch.where(keys[i] == want, d["logq"][i].double(), torch.full((n,), NEG, dtype=torch.float64, device=dev))
        out = torch.where(d["replayed"][:n].bool(), found, out)
    return out


def _probs(d, rows, V):
    """The rows' probabilities of every token, in 64 bits."""
    n, dev = rows.numel(), rows.device
    out = torch.zeros(n, V, dtype=torch.float64, device=dev)
    if d["logits"] is not None:
        z, T = d["logits"][rows].double(), _temps(d, d["logits"].shape[0], dev)[rows]
        zm, at, lt = _log_total(z, T)
        out = torch.exp((z - zm[:, None]) / torch.where(T > 0, T, torch.ones_like(T))[:, None] - lt[:, None])
        out = torch.where((T > 0)[:, None], out, torch.zeros_like(out).scatter_(1, at[:, None], 1.0))
    if d["offsets"] is not None:
        a, b = d["offsets"][rows], d["offsets"][rows + 1]
        b = torch.where(d["replayed"][rows].bool(), b, a)
        of = torch.repeat_interleave(torch.arange(n, device=dev), b - a)
        j = torch.arange(of.numel(), device=dev) - torch.cumsum(b - a, 0)[of] + b[of]
        held = torch.zeros_like(out)
        held[of, d["ids"][j].long()] = torch.exp(d["logq"][j].double())
        out = torch.where(d["replayed"][rows].bool()[:, None], held, out)
    return out


def _plain_verify(s):
    V, T, dev = s["V"], s["T"], s["cu_q"].device
    cu, R = s["cu_q"].long(), s["u_next"].numel()
    n = cu[1:] - cu[:-1]
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[r]
    last = i == n[r] - 1
    x = torch.where(last, torch.zeros_like(t), torch.roll(s["step_tokens"], -1).long())
    lp = _log_prob(s["target"], x, V)
    lq = torch.zeros_like(lp) if s["draft"] is None else _log_prob(s["draft"], x, V)
    ok = (s["u"].double() * torch.exp(lq) < torch.exp(lp)) & ~last
    stop = torch.where(ok, torch.full_like(i, 1 << 30), i)
    accepted = torch.full((R,), 1 << 30, dtype=torch.long, device=dev).scatter_reduce_(0, r, stop, "amin")
    live = n > 0
    accepted = torch.where(live, accepted, torch.zeros_like(accepted))
    at = (cu[:-1] + accepted).clamp(max=max(T - 1, 0))
    # what is left of the target at the first draft that was turned down, or the whole of it after the last
    p = _probs(s["target"], at, V)
    if s["draft"] is None:
        q = torch.zeros_like(p).scatter_(1, x[at][:, None], 1.0)
    else:
        q = _probs(s["draft"], at, V)
    q = torch.where((accepted < n - 1)[:, None], q, torch.zeros_like(q))
    left = (p - q).clamp(min=0)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, p)
    cdf = torch.cumsum(left, 1)
    new = torch.searchsorted(cdf, s["u_next"].double()[:, None] * cdf[:, -1:], right=True)[:, 0].clamp(max=V - 1)
    tokens = torch.where(i < accepted[r], x, torch.where(i == accepted[r], new[r], torch.full_like(x, -1)))
    new_lp = torch.log(p.gather(1, new[:, None])[:, 0])
    logq = torch.where(i < accepted[r], lp, torch.where(i == accepted[r], new_lp[r], torch.zeros_like(lp)))
    return dict(tokens=tokens.to(torch.int32), logq=logq.float(), accepted=accepted.to(torch.int32),
                keep_lens=(s["ctx_lens"] + torch.where(live, accepted + 1, accepted)).to(torch.int32))


def _mark(n_pages, table, lo, hi):
    """Which pages the entries lo <= j < hi of the rows name."""
    cols = torch.arange(table.shape[1], device=table.device)[None]
    named = (cols >= lo[:, None]) & (cols < hi[:, None])
    marks = torch.zeros(n_pages + 1, dtype=torch.bool, device=table.device)
    marks[torch.where(named, table.long(), torch.full_like(table, n_pages, dtype=torch.long)).view(-1)] = True
    return marks[:n_pages]


def _plain_release(s):
    page, n_pages, dev = s["page"], s["n_pages"], s["block_table"].device
    had, left = (s["kv_lens"].long() + page - 1) // page, (s["keep_lens"].long() + page - 1) // page
    zero = torch.zeros_like(had)
    freed = _mark(n_pages, s["block_table"], left, had) & ~_mark(n_pages, s["block_table"], zero, left)
    rank = torch.cumsum(freed, 0)
    used = s["free_used"].long() - rank[-1]
    pool = torch.cat([s["free_pages"], s["free_pages"][:1]])
    place = torch.where(freed, used + rank - 1, torch.full_like(rank, pool.numel() - 1))
    pool.scatter_(0, place, torch.arange(n_pages, device=dev, dtype=torch.int32))
    return dict(free_pages=pool[:-1], free_used=used.to(torch.int32))


def _plain_copies(kc, vc, src, dst, tokens):
    ok = src >= 0
    a, b = src[ok].long(), dst[ok].long()
    for c in (kc, vc):
        rows = c[:, a]
        if tokens is not None:
            new = torch.arange(c.shape[3], device=c.device)[None] < tokens[ok][:, None]
            rows = torch.where(new[None, :, None, :, None], rows, c[:, b])
        c[:, b] = rows


def _plain_fork(s):
    page, table = s["page"], s["block_table"].clone()
    dev, W, n = table.device, table.shape[1], s["lens"].long()
    full, part = n // page, n % page
    rank = torch.cumsum(part > 0, 0)
    fresh = s["free_pages"][(s["free_used"].long() + rank - 1).clamp(0, s["free_pages"].numel() - 1)]
    cols = torch.arange(W, device=dev)[None]
    theirs = table[s["parents"].long()]
    mine = torch.where(cols < full[:, None], theirs, torch.full_like(theirs, -1))
    mine = torch.where((cols == full[:, None]) & (part > 0)[:, None], fresh[:, None], mine)
    table[s["children"].long()] = mine
    kv = s["kv_lens"].clone()
    kv[s["children"].long()] = s["lens"]
    none = torch.full_like(fresh, -1)
    src = torch.where(part > 0, theirs.gather(1, full.clamp(max=W - 1)[:, None])[:, 0], none)
    dst = torch.where(part > 0, fresh, none)
    _plain_copies(s["k_cache"], s["v_cache"], src, dst, part)
    return dict(block_table=table, kv_lens=kv, src=src, dst=dst, tokens=part.to(torch.int32),
                free_used=(s["free_used"] + rank[-1]).to(torch.int32), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_compact(s):
    page, n_pages, dev = s["page"], s["n_pages"], s["block_table"].device
    had = [(s[k].long() + page - 1) // page for k in ("kv_lens", "prefix_lens")]
    live = _mark(n_pages, s["block_table"], torch.zeros_like(had[0]), had[0]) | \
        _mark(n_pages, s["prefix_table"], torch.zeros_like(had[1]), had[1])
    ids = torch.arange(n_pages, device=dev)
    n_live = live.sum()
    goes, hole = live & (ids >= n_live), ~live & (ids < n_live)
    cap = n_pages // 2
    src, dst = (torch.full((cap + 1,), -1, dtype=torch.long, device=dev).scatter_(
        0, torch.where(m, torch.cumsum(m, 0) - 1, torch.full_like(ids, cap)), ids)[:cap] for m in (goes, hole))
    to = torch.cat([ids, ids[:1]])
    to[torch.where(src >= 0, src, torch.full_like(src, n_pages))] = dst
    tables = []
    for name, h in (("block_table", had[0]), ("prefix_table", had[1])):
        t = s[name]
        named = torch.arange(t.shape[1], device=dev)[None] < h[:, None]
        tables.append(torch.where(named, to[t.long().clamp(min=0)].to(torch.int32), torch.full_like(t, -1)))
    _plain_copies(s["k_cache"], s["v_cache"], src, dst, None)
    return dict(block_table=tables[0], prefix_table=tables[1], src=src.to(torch.int32), dst=dst.to(torch.int32),
                free_pages=ids.to(torch.int32), free_used=n_live.to(torch.int32)[None], k_cache=s["k_cache"],
                v_cache=s["v_cache"])


def _plain_distill(s):
    z, off, ids = s["logits"], s["offsets"], s["ids"].long()
    N, dev, T, beta = z.shape[0], z.device, s["T"], s["beta"]
    row = torch.searchsorted(off, torch.arange(ids.numel(), device=dev), right=True) - 1
    zm = z.amax(1, keepdim=True).float()
    e = torch.exp((z.float() - zm) / T)
    total = e.sum(1, dtype=torch.float64)
    lp = (z[row, ids].double() - zm[row, 0]) / T - torch.log(total)[row]      # a divergence is a small difference of these
    pe = torch.exp(lp)
    e[row, ids] = 0                      # what is left is the rest of the vocabulary
    sums = lambda v: torch.zeros(N, dtype=v.dtype, device=dev).index_add_(0, row, v)  # noqa: E731
    if s["tail"]:
        lt = s["logq"].double()
        t = torch.exp(lt)
        t0 = (1 - sums(t)).clamp(min=2.0 ** -20)
        p0 = e.sum(1, dtype=torch.float64) / total
    else:
        y = s["logq"].double() / T
        top = torch.full((N,), NEG, dtype=torch.float64, device=dev).scatter_reduce_(0, row, y, "amax")
        lt = y - top[row] - torch.log(sums(torch.exp(y - top[row])))[row]
        t = torch.exp(lt)
        t0 = p0 = torch.zeros(N, dtype=torch.float64, device=dev)
    # f(P) of one outcome, and P f'(P) less what cancels in the gradient
    if s["kind"] == "forward":
        f = lambda t, lt, p, lp: (t * (lt - lp), -t)  # noqa: E731
    elif s["kind"] == "reverse":
        f = lambda t, lt, p, lp: (p * (lp - lt), p * (lp - lt))  # noqa: E731
    else:
        def f(t, lt, p, lp):
            lm = torch.log(beta * t + (1 - beta) * p)
            return beta * t * (lt - lm) + (1 - beta) * p * (lp - lm), (1 - beta) * p * (lp - lm)
    has = off.diff() > 0
    one, zero = torch.ones_like(p0), torch.zeros_like(p0)
    fe, ge = f(t, lt, pe, lp)
    rest = p0 > 0
    f0, g0 = f(t0, torch.log(torch.where(rest, t0, one)), p0, torch.log(torch.where(rest, p0, one)))
    f0, g0 = torch.where(rest, f0, zero), torch.where(rest, g0, zero)
    A = sums(ge) + g0
    coef = s["dloss"] / T * has
    d = e * (coef * (g0 / torch.where(rest, p0, one) - A) / total).float()[:, None]
    d[row, ids] = ((ge - pe * A[row]) * coef[row]).float()
    return dict(loss=torch.where(has, sums(fe) + f0, zero).float(), dlogits=d.to(z.dtype))


PLAIN = {"verify": _plain_verify, "release": _plain_release, "fork": _plain_fork, "compact": _plain_compact,
         "distill": _plain_distill}


# ---- the library's calls ---------------------------------------------------------------

def _own_verify(s):
    import lm_head_gb300 as rh
    k = s["keep"]
    if "target" not in k:
        k["target"] = rh.Dist(**s["target"])
        k["draft"] = None if s["draft"] is None else rh.Dist(**s["draft"])
    o = rh.rl_verify(s["step_tokens"], s["cu_q"], s["u"], s["u_next"], k["target"], k["draft"], vocab=s["V"],
                     ctx_lens=s["ctx_lens"], out=k.get("out"))
    k["out"] = o
    return dict(tokens=o.tokens, logq=o.logq, accepted=o.accepted, keep_lens=o.keep_lens)


def _own_release(s):
    import lm_head_gb300 as rh
    k = s["keep"]
    o = rh.rl_page_release(s["kv_lens"], s["keep_lens"], s["block_table"], s["free_pages"], s["free_used"],
                           page_size=s["page"], n_pages=s["n_pages"], out=k.get("out"))
    k["out"] = o
    return dict(free_pages=s["free_pages"], free_used=o.free_used)


def _own_fork(s):
    import lm_head_gb300 as rh
    k = s["keep"]
    o = rh.rl_page_fork(s["parents"], s["children"], s["lens"], s["kv_lens"], s["block_table"], s["free_pages"],
                        s["free_used"], page_size=s["page"], n_pages=s["n_pages"], out=k.get("out"))
    k["out"] = o
    rh.rl_page_copy(o.src, o.dst, s["k_cache"], s["v_cache"], tokens=o.tokens, status=o.status)
    return dict(block_table=s["block_table"], kv_lens=s["kv_lens"], src=o.src, dst=o.dst, tokens=o.tokens,
                free_used=o.free_used, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_compact(s):
    import lm_head_gb300 as rh
    k = s["keep"]
    o = rh.rl_page_compact(s["kv_lens"], s["block_table"], page_size=s["page"], n_pages=s["n_pages"],
                           prefix_lens=s["prefix_lens"], prefix_table=s["prefix_table"], out=k.get("out"))
    k["out"] = o
    rh.rl_page_copy(o.src, o.dst, s["k_cache"], s["v_cache"], status=o.status)
    return dict(block_table=o.block_table, prefix_table=o.prefix_table, src=o.src, dst=o.dst, free_pages=o.free_pages,
                free_used=o.free_used, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_distill(s):
    import lm_head_gb300 as rh
    k = s["keep"]
    if "params" not in k:
        k["params"] = rh.DistillParams(kind=s["kind"], tail=s["tail"], temperature=s["T"], beta=s["beta"])
    o, d = rh.rl_distill_fwd_bwd(s["logits"], s["offsets"], s["ids"], s["logq"], s["dloss"], k["params"], out=k.get("out"),
                                 dlogits=k.get("d"))
    k["out"], k["d"] = o, d
    return dict(loss=o.loss, dlogits=d)


OWN = {"verify": _own_verify, "release": _own_release, "fork": _own_fork, "compact": _own_compact, "distill": _own_distill}


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "verify":
        T, e = c["R"] * (c["q_min"] + c["q_max"]) / 2, ELEM[c["dtype"]]
        whole = {"dense": 1.0, "mixed": 0.5}
        rows = whole.get(c["target"], 0) * T + whole.get(c["draft"], 0) * max(T - c["R"], 0)
        held = 16 * (T if c["target"] != "dense" else 0) + 16 * (T if c["draft"] in ("rows", "mixed") else 0)
        return {"bytes": rows * c["V"] * e + 8 * held + 16 * T + 16 * c["R"], "flops": 3 * rows * c["V"]}
    if c["op"] == "release":
        pages = c["R"] * (c["len_max"] / 2 / c["page"] + 0.5)
        given = pages / 2 if c["drop"] < 0 else c["R"] * c["drop"] / 2 / c["page"]
        return {"bytes": 8 * c["R"] + 4 * pages + 4 * given, "flops": 0}
    token = 2 * c["L"] * c["Hkv"] * c["D"] * ELEM[c["dtype"]] if "L" in c else 0
    if c["op"] == "fork":
        full = c["len_max"] / 2 / c["page"]
        part = min(c["page"], c["len_max"]) / 2
        return {"bytes": c["C"] * (20 + 8 * full) + 2 * token * c["C"] * part, "flops": 0}
    if c["op"] == "compact":
        pages = (c["R"] + c["G"]) * (c["len_max"] / 2 / c["page"] + 0.5)
        moved = pages * (1 - 1 / c["spread"])
        return {"bytes": 8 * pages + 4 * pages * c["spread"] + 8 * moved + 2 * token * c["page"] * moved, "flops": 0}
    n = c["N"] * c["V"]
    return {"bytes": 2 * n * ELEM[c["dtype"]] + c["N"] * (8 * (c["k_min"] + c["k_max"]) / 2 + 16), "flops": 4 * n}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_row(d, t, V):
    """One row's distribution over the vocabulary."""
    if d["offsets"] is not None and bool(d["replayed"][t]):
        a, b = int(d["offsets"][t]), int(d["offsets"][t + 1])
        p = torch.zeros(V, dtype=torch.float64, device="cuda")
        p[d["ids"][a:b].long()] = d["logq"][a:b].double().exp()
        return p
    z = d["logits"][t].double()
    T = 1.0 if d["temperature"] is None else float(d["temperature"][t])
    if T == 0:
        p = torch.zeros_like(z)
        p[int((z == z.max()).nonzero()[0, 0])] = 1
        return p
    return torch.softmax(z / T, 0)


def _exact_verify(s):
    """The definition request by request, token by token."""
    V, cu, R = s["V"], s["cu_q"].tolist(), s["u_next"].numel()
    step, u, u_next, ctx = (s[n].tolist() for n in ("step_tokens", "u", "u_next", "ctx_lens"))
    tokens, logq = [-1] * s["T"], torch.zeros(s["T"], dtype=torch.float64)
    accepted, keep = [0] * R, list(ctx)
    for r in range(R):
        n = cu[r + 1] - cu[r]
        if n == 0:
            continue
        left = None
        for i in range(n):
            t = cu[r] + i
            p = _exact_row(s["target"], t, V)
            left = p
            if i == n - 1:
                break
            x = step[t + 1]
            if s["draft"] is None:
                q = torch.zeros_like(p)
                q[x] = 1
            else:
                q = _exact_row(s["draft"], t, V)
            if u[t] * float(q[x]) < float(p[x]):
                tokens[t], logq[t] = x, math.log(float(p[x]))
                accepted[r] += 1
                continue
            over = torch.relu(p - q)
            left = over if float(over.sum()) > 0 else p
            break
        c = left.cumsum(0)
        y = int((c <= u_next[r] * c[-1]).sum().clamp(max=V - 1))
        tokens[t], logq[t] = y, math.log(float(p[y]))
        keep[r] = ctx[r] + accepted[r] + 1
    i32 = torch.int32
    return dict(tokens=torch.tensor(tokens, dtype=i32), logq=logq, accepted=torch.tensor(accepted, dtype=i32),
                keep_lens=torch.tensor(keep, dtype=i32))


def _exact_distill(s):
    """Every outcome's probabilities written out, a row at a time; the gradient as the logits' softmax maps it."""
    z, T, beta = s["logits"], s["T"], s["beta"]
    N = z.shape[0]
    off = s["offsets"].tolist()
    loss, grad = torch.zeros(N, dtype=torch.float64), torch.zeros(z.shape, dtype=torch.float64, device="cuda")
    weight = s["dloss"].tolist()
    for r in range(N):
        a, b = off[r], off[r + 1]
        if a == b:
            continue
        ids = s["ids"][a:b].long()
        x = z[r].double() / T
        P = torch.softmax(x, 0)
        lP = torch.log_softmax(x, 0)
        out = torch.ones(z.shape[1], dtype=torch.bool, device="cuda")
        out[ids] = False
        y = s["logq"][a:b].double()
        if s["tail"]:
            rest = P[out].sum()
            t = torch.cat([y.exp(), (1 - y.exp().sum()).clamp(min=2.0 ** -20)[None]])
            p, lp = torch.cat([P[ids], rest[None]]), torch.cat([lP[ids], torch.log(rest)[None]])
            lt = torch.cat([y, torch.log(t[-1:])])
        else:
            t, lt = torch.softmax(y / T, 0), torch.log_softmax(y / T, 0)
            p, lp = P[ids], lP[ids]
        if s["kind"] == "forward":
            v, dv = (t * (lt - lp)).sum(), -t / p
        elif s["kind"] == "reverse":
            v, dv = (p * (lp - lt)).sum(), lp - lt + 1
        else:
            lm = torch.log(beta * t + (1 - beta) * p)
            v, dv = (beta * t * (lt - lm) + (1 - beta) * p * (lp - lm)).sum(), (1 - beta) * (lp - lm)
        g = torch.full_like(P, float(dv[-1]) if s["tail"] else 0.0)
        g[ids] = dv[:b - a]
        loss[r] = v
        grad[r] = P * (g - (P * g).sum()) * (weight[r] / T)
    return dict(loss=loss, dlogits=grad)


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return _exact_verify(prepare(case, seed))
    if c["op"] == "distill":
        return _exact_distill(prepare(case, seed))
    return None             # page lists and copies compute no numbers of their own
