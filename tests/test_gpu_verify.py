"""Verification of drafts against the definition in 64 bits: every token equal unless a random number lies within the
sums' accuracy of a border."""
import math

import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from verify_ref import Side, verify_reference

pytestmark = pytest.mark.gpu
OFFSETS, ID_RANGE, LOGQ, EMPTY, ORDER, NONFINITE, LENGTHS, KNOB = 0x1, 0x2, 0x4, 0x20, 0x40, 0x100, 0x400, 0x2000
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
MARGIN = 2.0 ** -33         # sums are carried to about 2^-36 of the whole; the reference's own are good to 2^-48


def cuda(x, dtype):
    return None if x is None else torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda()


class Half:
    """One side's distributions, for the reference and for the call."""

    def __init__(self, V, z=None, temp=None, ids=None, lq=None, rep=None, rows=None, pad=0):
        z64 = None if z is None else z.double().numpy()
        self.side = Side(V, z64, temp, ids, lq, rep, rows)
        d = dict(temperature=cuda(temp, torch.float32), replayed=cuda(rep, torch.uint8), rows=cuda(rows, torch.int32))
        if z is not None:
            buf = torch.full((z.shape[0] * (V + pad) + 1,), 9.0, dtype=z.dtype, device="cuda")
            v = buf[1 if pad else 0:].as_strided((z.shape[0], V), (V + pad, 1))
            v.copy_(z)
            d["logits"] = v
        if ids is not None:
            d["offsets"] = cuda(np.concatenate([[0], np.cumsum([len(x) for x in ids])]), torch.int64)
            cat = lambda a: np.concatenate([np.asarray(x, float) for x in a]) if len(a) else np.zeros(0)  # noqa: E731
            d["ids"], d["logq"] = cuda(cat(ids), torch.int32), cuda(cat(lq), torch.float32)
        self.dist = rh.Dist(**d)


def support_of(z, temp, rng, most):
    """Truncated rows: the largest few of each, renormalised in fp32."""
    ids, lq = [], []
    for r in range(z.shape[0]):
        T = float(temp[r]) if temp is not None and temp[r] > 0 else 1.0
        n = int(rng.integers(1, most + 1))
        x = z[r].double().numpy() / T
        i = np.sort(np.argsort(-x, kind="stable")[:n])
        lp = x[i] - x[i].max()
        ids.append(i)
        lq.append((lp - math.log(np.exp(lp).sum())).astype(np.float32))
    return ids, lq


def case(R, q_min, q_max, V, target="dense", draft="dense", dtype=("fp32", "fp32"), temps=False, seed=0, near=0.7, scale=2.0, pad=0,
         maps=False, most=40, u=None):
    rng = np.random.default_rng(seed * 1009 + V)
    n = rng.integers(q_min, q_max + 1, R)
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1])
    g = torch.Generator().manual_seed(seed + V)
    z = torch.randn(max(T, 1), V, generator=g) * scale
    zd = 0.9 * z + near * torch.randn(max(T, 1), V, generator=g)
    halves = []
    order = rng.permutation(max(T, 1)) if maps else None       # row t of the step is row order[t] of what is held
    for x, form, dt in ((z, target, dtype[0]), (zd, draft, dtype[1])):
        if form == "sure":
            halves.append(None)
            continue
        x = x.to(DT[dt])
        temp = np.where(rng.random(max(T, 1)) < 0.15, 0, rng.uniform(0.5, 1.5, max(T, 1))).astype(np.float32) if temps else None
        ids = lq = rep = None
        if form != "dense":
            ids, lq = support_of(x, temp, rng, min(most, V))
            rep = (rng.random(max(T, 1)) < 0.5).astype(np.uint8) if form == "mixed" else None
        if maps:
            inv = np.argsort(order)
            x, temp = x[inv], None if temp is None else temp[inv]
            ids, lq = (None, None) if ids is None else ([ids[i] for i in inv], [lq[i] for i in inv])
            rep = None if rep is None else rep[inv]
        halves.append(Half(V, None if form == "rows" else x, temp, ids, lq, rep, order, pad))
    step = rng.integers(0, V, T)
    for t in range(1, T):               # candidates drawn from the drafts
        if halves[1] is None:
            step[t] = int(torch.argmax(zd[t - 1])) if rng.random() < 0.7 else step[t]
        else:
            p = np.exp(halves[1].side.log_probs(t - 1))
            step[t] = rng.choice(V, p=p / p.sum())
    f = lambda k: (rng.integers(0, 1 << 24, k) / 2.0 ** 24).astype(np.float32)  # noqa: E731
    return dict(step=step, cu=cu, u=f(T) if u is None else np.full(T, u, np.float32), un=f(R), target=halves[0], draft=halves[1], V=V,
                ctx=rng.integers(0, 1000, R))


def call(c, **kw):
    return rh.rl_verify(cuda(c["step"], torch.int32), cuda(c["cu"], torch.int32), cuda(c["u"], torch.float32),
                        cuda(c["un"], torch.float32), c["target"].dist, None if c["draft"] is None else c["draft"].dist,
                        vocab=c["V"], ctx_lens=cuda(c["ctx"], torch.int32), **kw)


def check(c, bits=0, skips=0):
    with np.errstate(all="ignore"):
        ref = verify_reference(c["step"], c["cu"], c["u"], c["un"], c["target"].side, None if c["draft"] is None else c["draft"].side,
                               c["ctx"])
    o = call(c)
    for again in range(2):
        tokens, logq, acc, keep = (x.cpu().numpy() for x in (o.tokens, o.logq, o.accepted, o.keep_lens))
        left_out = 0
        seen = np.zeros(len(c["step"]), bool)
        for r in range(len(c["cu"]) - 1):
            a, b = int(c["cu"][r]), int(c["cu"][r + 1])
            if not 0 <= a <= b <= len(c["step"]):
                a = b = 0
            seen[a:b] = True
            if ref["margin"][r] < MARGIN:
                left_out += 1
                continue
            assert acc[r] == ref["accepted"][r] and keep[r] == ref["keep_lens"][r], r
            np.testing.assert_array_equal(tokens[a:b], ref["tokens"][a:b], err_msg=str(r))
            # ln p: roundings of its own size, and of an accepted token's total of fp32 exponentials: 2^-22 each, two roundings of
            # an argument of at most 20 where it counts (2^20 weights of 2^-20 are as much as the largest), 20 in its chunk's
            # scale, and 60 additions: 2^-22 + (20 + 20 + 60) 2^-24
            want = ref["logq"][a:b]
            with np.errstate(all="ignore"):
                ok = (np.abs(logq[a:b] - want) <= 2.0 ** -22 * np.abs(want) + 104 * 2.0 ** -24) | (logq[a:b] == want)
            assert ok.all(), (r, logq[a:b], want)
        assert (tokens[~seen] == -1).all() and (logq[~seen] == 0).all()
        assert left_out <= skips, left_out
        assert o.status_bits() == bits, hex(o.status_bits())
        o.ws.fill_(255)
        o = call(c, out=o)
    return ref, o


FORMS = [(t, d) for t in ("dense", "rows", "mixed") for d in ("dense", "rows", "mixed", "sure")]


@pytest.mark.parametrize("target,draft", FORMS)
@pytest.mark.parametrize("V", [1, 2, 5, 128, 129, 1000, 4103])
def test_against_the_definition(target, draft, V):
    for i, (dt, temps) in enumerate(((("fp32", "bf16"), True), (("fp16", "fp32"), False), (("bf16", "bf16"), True))):
        ref, _ = check(case(40, 0, 7, V, target, draft, dt, temps, seed=i))
        if V > 100 and draft != "sure":
            assert 0 < ref["accepted"].sum() < 200          # drafts are taken and turned down


@pytest.mark.parametrize("target,draft", [("dense", "dense"), ("mixed", "rows"), ("rows", "dense"), ("dense", "sure")])
@pytest.mark.parametrize("R,V", [(1, 151936), (3, 50257), (17, 32768), (300, 777)])
def test_sizes(target, draft, R, V):
    check(case(R, 1, 6, V, target, draft, ("bf16", "fp32"), True, seed=R, most=500))


@pytest.mark.parametrize("pad", [0, 1, 3, 4])
def test_strides_and_row_maps(pad):
    for dt in (("fp32", "fp16"), ("bf16", "fp32")):
        check(case(20, 0, 5, 1001, "dense", "dense", dt, True, seed=pad, pad=pad))
        check(case(20, 1, 5, 1004, "mixed", "mixed", dt, True, seed=pad, pad=pad, maps=True))


def test_one_row_requests_are_plain_sampling():
    c = case(64, 1, 1, 5003, "dense", "dense", temps=True, seed=3)
    ref, _ = check(c)
    assert not ref["accepted"].any()


def test_long_requests():
    check(case(3, 60, 90, 300, "dense", "dense", near=0.05, seed=4))
    check(case(2, 300, 400, 64, "rows", "rows", near=0.02, seed=5))


@pytest.mark.parametrize("form", ["dense", "rows"])
def test_the_same_distribution_accepts_everything(form):
    """p = q: u q < p for every u below 1, the largest float below 1 among them."""
    c = case(12, 2, 6, 2000, form, form, near=0.0, seed=6, u=1 - 2.0 ** -24)
    c["draft"] = c["target"]
    for t in range(1, len(c["step"])):          # candidates with a probability
        c["step"][t] = int(np.argmax(c["target"].side.log_probs(t - 1)))
    ref, o = check(c)
    assert (ref["accepted"] == np.diff(c["cu"]) - 1).all()


def test_supports_that_do_not_meet():
    V, T = 100, 6
    ids = [np.arange(10)] * T
    other = [np.arange(50, 60)] * T
    lq = [np.full(10, math.log(0.1), np.float32)] * T
    c = dict(step=np.full(T, 55), cu=np.array([0, 3, 6]), u=np.zeros(T, np.float32), un=np.array([0.0, 0.95], np.float32), V=V,
             ctx=np.zeros(2, int), target=Half(V, ids=ids, lq=lq), draft=Half(V, ids=other, lq=lq))
    _, o = check(c)
    assert o.accepted.tolist() == [0, 0] and o.tokens[0] == 0 and o.tokens[3] == 9


def test_nothing_left_falls_back_to_the_target():
    """A draft row that lies above the target's everywhere (its mass is above 1): the draw is from p itself."""
    V = 50
    ids = [np.arange(10)] * 2
    lq = np.log(np.arange(1, 11) / 55.0).astype(np.float32)
    hi = np.minimum(lq + 0.5, 0).astype(np.float32)
    c = dict(step=np.array([0, 9]), cu=np.array([0, 2]), u=np.array([0.99, 0], np.float32), un=np.array([0.6], np.float32), V=V,
             ctx=np.zeros(1, int), target=Half(V, ids=ids, lq=[lq] * 2), draft=Half(V, ids=ids, lq=[hi] * 2))
    ref, o = check(c)
    assert ref["accepted"][0] == 0 and int(o.tokens[0]) == 7
    # and with logits on both sides that are the same, a candidate outside the vocabulary
    z = torch.randn(2, V)
    c = dict(c, target=Half(V, z), draft=Half(V, z), step=np.array([0, V]))
    with np.errstate(all="ignore"):
        ref = verify_reference(c["step"], c["cu"], c["u"], c["un"], c["target"].side, c["draft"].side, c["ctx"])
    o = call(c)
    assert o.status_bits() == ID_RANGE and int(o.accepted[0]) == 0 and int(o.tokens[0]) == ref["tokens"][0]


def test_random_numbers_next_to_the_border():
    """u one float below and above p / q, where 64 bits tell them apart and 32 would not."""
    rng = np.random.default_rng(8)
    V, T = 3000, 80
    z = torch.randn(T, V, generator=torch.Generator().manual_seed(8)) * 2
    zd = z + 0.5 * torch.randn(T, V, generator=torch.Generator().manual_seed(9))
    for tf, df in (("dense", "dense"), ("dense", "rows"), ("rows", "dense"), ("rows", "rows"), ("dense", "sure")):
        halves = []
        for x, f in ((z, tf), (zd, df)):
            if f == "sure":
                halves.append(None)
            elif f == "dense":
                halves.append(Half(V, x))
            else:
                ids, lq = support_of(x, None, rng, 200)
                halves.append(Half(V, ids=ids, lq=lq))
        step, u = np.zeros(T, int), np.zeros(T, np.float32)
        for t in range(0, T, 2):
            lp = halves[0].side.log_probs(t)
            lq = np.zeros(V) if halves[1] is None else halves[1].side.log_probs(t)
            ok = np.flatnonzero((lp > -np.inf) & (lq > lp) & (lq > -np.inf))
            x = int(rng.choice(ok)) if len(ok) else 0
            b = np.float32(math.exp(min(lp[x] - lq[x], 0))) if len(ok) else np.float32(0.5)
            step[t + 1], u[t] = x, np.nextafter(b, np.float32(t % 4 // 2 * 2 - 1 + 1e-9), dtype=np.float32) if t % 8 < 4 else b
        c = dict(step=step, cu=np.arange(0, T + 1, 2), u=np.minimum(u, np.float32(1 - 2.0 ** -24)), V=V, ctx=np.zeros(T // 2, int),
                 un=rng.random(T // 2).astype(np.float32), target=halves[0], draft=halves[1])
        check(c, skips=2)


def test_wide_flat_and_steep_rows():
    """The largest vocabulary with equal logits, a likely token over a long flat tail, logits of size 1e5, almost all masked."""
    V = 1 << 20
    g = torch.Generator().manual_seed(2)
    z = torch.zeros(4, V)
    z[1, 77] = 12.0
    z[2] = torch.randn(V, generator=g) * 3e4
    z[3] = float("-inf")
    z[3, [5, V - 1]] = 1.0
    zd = z + torch.randn(4, V, generator=g)
    zd[3] = z[3]
    step = np.array([0, 9, 0, 77, 0, int(z[2].argmax()), 0, V - 1])
    z2, zd2 = z.repeat_interleave(2, 0), zd.repeat_interleave(2, 0)
    for un in (0.3, 0.999, 0.0):
        c = dict(step=step, cu=np.arange(0, 9, 2), u=np.full(8, 0.9, np.float32), un=np.full(4, un, np.float32), V=V, ctx=np.zeros(4, int),
                 target=Half(V, z2), draft=Half(V, zd2))
        check(c, skips=0)
        check(dict(c, draft=None))
        # whole targets under a draft's support rows
        ids = [np.array([3, 9, 77, V - 1])] * 8
        lq = [np.log(np.array([0.1, 0.2, 0.3, 0.4])).astype(np.float32)] * 8
        check(dict(c, draft=Half(V, ids=ids, lq=lq)))


def test_temperatures():
    T, V = 8, 600
    z = torch.randn(T, V, generator=torch.Generator().manual_seed(1))
    z[3, 100] = z[3, 7] = z[3].max() + 1            # equal largest logits: the lowest index
    temp = np.array([0, 1e-30, 1e30, 0, 0.01, 100, 1, 0], np.float32)
    step = np.zeros(T, int)
    for t in range(T - 1):
        step[t + 1] = int(z[t].argmax())
    step[4] = 7
    c = dict(step=step, cu=np.arange(T + 1), u=np.full(T, 0.5, np.float32), un=np.full(T, 0.5, np.float32), V=V, ctx=np.zeros(T, int),
             target=Half(V, z, temp), draft=Half(V, z, temp[::-1].copy()))
    check(c, skips=1)           # (600 weights of 1 at T = 1e30: row 2's number is on a border)
    check(dict(c, cu=np.array([0, 8]), un=c["un"][:1], ctx=c["ctx"][:1]))
    for bad in (-1.0, float("nan"), float("inf"), 1e-38):
        t2 = temp.copy()
        t2[6] = bad
        c2 = dict(c, target=Half(V, z, t2), cu=np.array([0, 6, 8]), un=c["un"][:2], ctx=c["ctx"][:2], draft=None)
        c2["target"].side.temp = np.where(np.arange(T) == 6, 0, temp)
        c2["target"].side.kept.clear()
        check(c2, KNOB)


def test_bad_inputs():
    base = lambda **kw: case(6, 2, 4, 500, "mixed", "mixed", temps=False, seed=12, **kw)  # noqa: E731

    def run(change, bits, skips=6):
        c = base()
        change(c)
        o = call(c)
        assert o.status_bits() == bits, (hex(o.status_bits()), hex(bits))
        return o
    check(base())

    def put(c, name, i, v):
        c[name] = c[name].copy()
        c[name][i] = v
    # offsets of requests
    c = base()
    put(c, "cu", 2, c["cu"][3] + 1)
    check(c, LENGTHS)
    c = base()
    put(c, "cu", 0, -1)
    check(c, LENGTHS)
    c = base()
    put(c, "cu", 6, c["cu"][6] + 5)
    check(c, LENGTHS)
    # candidates
    for v in (-1, 500, 1 << 30):
        c = base()
        put(c, "step", 1, v)
        check(c, ID_RANGE)
    # random numbers
    for v, as_ in ((-0.5, 0.0), (1.0, 1 - 2.0 ** -24), (float("nan"), 0.0)):
        c = base()
        put(c, "u", 0, as_)
        put(c, "un", 1, as_)
        ref, want = check(c)
        put(c, "u", 0, v)
        put(c, "un", 1, v)
        o = call(c)
        assert o.status_bits() == KNOB and torch.equal(o.tokens, want.tokens)
    # logits that are not numbers count as -inf
    for v in (float("nan"), float("inf")):
        c = case(3, 3, 3, 500, "dense", "dense", seed=13)
        for h in (c["target"], c["draft"]):
            h.dist.logits[:, 17:29] = v
            h.side.z[:, 17:29] = -np.inf
            h.side.kept.clear()
        check(c, NONFINITE)
    # rows without a token
    c = case(3, 3, 3, 500, "dense", "dense", seed=14)
    for h, t in ((c["target"], 0), (c["draft"], 3)):
        h.dist.logits[t] = float("-inf")
        h.side.z[t] = -np.inf
        h.side.kept.clear()
    ref, o = check(c, EMPTY)
    assert int(o.accepted[0]) == 0 and int(o.tokens[0]) == -1 and float(o.logq[0]) == -math.inf
    # support rows
    c = case(2, 2, 2, 500, "rows", "rows", seed=15)
    n = c["target"].dist.ids.numel()
    for name, v, bits in (("ids", 500, ID_RANGE), ("ids", -3, ID_RANGE), ("logq", float("nan"), LOGQ), ("logq", 0.5, LOGQ),
                          ("offsets", -1, OFFSETS), ("offsets", n + 1, OFFSETS)):
        c = case(2, 1, 1, 500, "rows", "rows", seed=15)
        getattr(c["target"].dist, name)[0] = v
        o = call(c)
        assert o.status_bits() & bits
    c = case(2, 1, 1, 500, "rows", "rows", seed=16)
    c["target"].dist.ids[:2] = c["target"].dist.ids[:2].flip(0).clone()
    if int(c["target"].dist.offsets[1]) > 1:
        assert call(c).status_bits() & ORDER
    # row maps
    c = case(4, 2, 2, 300, "dense", "dense", seed=17, maps=True)
    for v in (-1, 8, 1 << 30):
        c["target"].dist.rows[2] = v
        o = call(c)
        assert o.status_bits() & OFFSETS and int(o.accepted[1]) == 0 and int(o.tokens[2]) == -1


def test_no_requests_and_no_rows():
    c = case(3, 0, 0, 100, "dense", "dense")
    o = call(c)
    assert o.accepted.tolist() == [0, 0, 0] and o.keep_lens.tolist() == c["ctx"].tolist() and o.status_bits() == 0
    c = case(2, 2, 2, 100, "dense", "dense")
    c.update(cu=np.array([0]), un=np.zeros(0), ctx=np.zeros(0))
    o = call(c)
    assert (o.tokens == -1).all() and o.status_bits() == 0


def test_more_rows_than_are_looked_up():
    """A step of more rows than a block keeps a list of."""
    rng = np.random.default_rng(2)
    R, n, V, kept = 9000, 4, 24, 40
    z = torch.randn(kept, V, generator=torch.Generator().manual_seed(2)) * 2
    zd = z + 0.3 * torch.randn(kept, V, generator=torch.Generator().manual_seed(3))
    rows = rng.integers(0, kept, R * n)
    c = dict(step=rng.integers(0, V, R * n), cu=np.arange(0, R * n + 1, n), u=(rng.integers(0, 1 << 24, R * n) / 2.0 ** 24).astype(np.float32),
             un=(rng.integers(0, 1 << 24, R) / 2.0 ** 24).astype(np.float32), V=V, ctx=np.zeros(R, int), target=Half(V, z, rows=rows),
             draft=Half(V, zd, rows=rows))
    ref, _ = check(c, skips=2)
    assert ref["accepted"].sum() > R / 2


@pytest.mark.parametrize("R", [2000, 2100])
def test_mixed_rows_about_as_many_as_are_listed(R):
    """Rows that may be support rows are listed up to a number of them: steps of 8000 and 8400 rows."""
    rng = np.random.default_rng(R)
    n, V, kept = 4, 40, 60
    z = torch.randn(kept, V, generator=torch.Generator().manual_seed(2)) * 2
    zd = z + 0.3 * torch.randn(kept, V, generator=torch.Generator().manual_seed(3))
    halves = []
    for x in (z, zd):
        ids, lq = support_of(x, None, rng, 20)
        halves.append(Half(V, x, ids=ids, lq=lq, rep=(rng.random(kept) < 0.5).astype(np.uint8), rows=rng.integers(0, kept, R * n)))
    c = dict(step=rng.integers(0, V, R * n), cu=np.arange(0, R * n + 1, n), u=(rng.integers(0, 1 << 24, R * n) / 2.0 ** 24).astype(np.float32),
             un=(rng.integers(0, 1 << 24, R) / 2.0 ** 24).astype(np.float32), V=V, ctx=np.zeros(R, int), target=halves[0], draft=halves[1])
    ref, _ = check(c, skips=2)
    assert ref["accepted"].sum() > R / 4


def test_tokens_are_the_targets_samples():
    """Over many requests with one draft each the new tokens at the first place follow p: six deviations of each count."""
    V, R = 12, 200000
    g = torch.Generator().manual_seed(3)
    z, zd = torch.randn(1, V, generator=g), torch.randn(1, V, generator=g)
    rng = np.random.default_rng(5)
    x = rng.choice(V, R, p=torch.softmax(zd[0].double(), 0).numpy())
    step = np.zeros(2 * R, int)
    step[1::2] = x
    zero = np.zeros(2 * R, int)
    c = dict(step=step, cu=np.arange(0, 2 * R + 1, 2), u=rng.random(2 * R).astype(np.float32).clip(max=1 - 2.0 ** -24),
             un=rng.random(R).astype(np.float32).clip(max=1 - 2.0 ** -24), V=V, ctx=np.zeros(R, int),
             target=Half(V, z, rows=zero), draft=Half(V, zd, rows=zero))
    o = call(c)
    first = np.bincount(o.tokens[::2].cpu().numpy(), minlength=V)
    p = torch.softmax(z[0].double(), 0).numpy()
    assert (np.abs(first - R * p) <= 6 * np.sqrt(R * p * (1 - p))).all()
    share = np.minimum(p, torch.softmax(zd[0].double(), 0).numpy()).sum()
    assert abs(float(o.accepted.float().mean()) - share) <= 6 * math.sqrt(share * (1 - share) / R)


def test_graphs_and_streams():
    c = case(30, 1, 5, 5003, "mixed", "rows", ("bf16", "bf16"), True, seed=20)
    args = lambda: (cuda(c["step"], torch.int32), cuda(c["cu"], torch.int32), cuda(c["u"], torch.float32),  # noqa: E731
                    cuda(c["un"], torch.float32), c["target"].dist, c["draft"].dist)
    a = args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = rh.rl_verify(*a, vocab=c["V"], stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rh.rl_verify(*a, vocab=c["V"], out=o)
    a[2].mul_(0.3)
    a[3].mul_(0.5)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want = rh.rl_verify(*a, vocab=c["V"])
    for x, y in ((o.tokens, want.tokens), (o.logq, want.logq), (o.accepted, want.accepted)):
        assert torch.equal(x, y)
    t = torch.cuda.Stream()
    t.wait_stream(torch.cuda.current_stream())
    res = [rh.rl_verify(*a, vocab=c["V"], stream=x) for x in (s, t) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(r.tokens, want.tokens) and torch.equal(r.logq, want.logq) for r in res)


def test_lengths_in_place():
    c = case(9, 0, 4, 200, "dense", "sure", seed=21)
    ref, o = check(c)
    ctx = cuda(c["ctx"], torch.int32)
    o.keep_lens = ctx
    rh.rl_verify(cuda(c["step"], torch.int32), cuda(c["cu"], torch.int32), cuda(c["u"], torch.float32), cuda(c["un"], torch.float32),
                 c["target"].dist, None, vocab=c["V"], ctx_lens=ctx, out=o)
    assert ctx.tolist() == ref["keep_lens"].tolist()
