"""Distillation from a teacher's top tokens against the definition in 64 bits, against differences of its own
loss, and on rows that are empty, masked, unaligned, in place or not valid."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from distill_ref import distill_reference, rest_error

pytestmark = pytest.mark.gpu
ID_RANGE, OFFSETS, LOGQ, ROW_ORDER, NONFINITE = 0x2, 0x1, 0x4, 0x40, 0x100
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}      # half a step, relative
LEAST = {"fp32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -25}


def make(N, V, dtype, k, T=1.0, tail=True, seed=0, scale=2.0, pad=0, shift=0):
    """Logits in a buffer with `pad` elements after each row, `shift` before the first; a teacher near them; k: sizes of the rows."""
    g = torch.Generator().manual_seed(seed * 31 + V)
    z = (torch.randn(N, V, generator=g) * scale).to(DT[dtype])
    teacher = z.double() + 0.7 * torch.randn(N, V, generator=g, dtype=torch.float64)
    lq = torch.log_softmax(teacher / T, 1) if tail else teacher
    ids, q = [], []
    for r in range(N):
        n = int(k[r])
        pick = torch.topk(teacher[r], n).indices if r % 2 else torch.randperm(V, generator=g)[:n]
        pick = torch.sort(pick).values
        ids.append(pick)
        q.append(lq[r, pick])
    off = torch.tensor([0] + [len(x) for x in ids]).cumsum(0)
    buf = torch.full((shift + N * (V + pad),), 7.0, dtype=DT[dtype], device="cuda")
    v = buf[shift:].as_strided((N, V), (V + pad, 1), buf.storage_offset() + shift)
    v.copy_(z)
    dl = torch.rand(N, generator=g) + 0.5
    if N > 2:
        dl[1] = 0.0
    return dict(z=v, buf=buf, off=off.cuda(), ids=torch.cat(ids).to(torch.int32).cuda(), q=torch.cat(q).float().cuda(),
                dl=dl.cuda())


def reference(c, p):
    return distill_reference(c["z"].float().cpu().numpy(), c["off"].cpu().numpy(), c["ids"].cpu().numpy(), c["q"].cpu().numpy(),
                             c["dl"].cpu().numpy(), p.kind, p.tail, p.temperature, p.beta)


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    inf = ~np.isfinite(want)
    assert np.array_equal(got[inf], want[inf], equal_nan=True), what
    bad = ~(np.abs(got - want) <= tol) & ~inf
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], tol[bad][:4])


def check(c, p, dtype, grad=None, spread=None):
    """Forward and backward in one call, then in two."""
    ref = reference(c, p)
    N, V = c["z"].shape
    eps = rest_error(p.temperature, V, spread if spread is not None else 24.0)
    # pairs of floats carry 2^-40 of terms that are at most 100 each
    t_loss = 1.1 * eps * ref["e_loss"] + 2.0 ** -23 * np.abs(ref["loss"]) + 2.0 ** -40 * 100 + 1e-12
    # (a gradient has three factors of that error at most: the exponential, the total and A)
    t_grad = 3.3 * eps * ref["e_grad"] + (HALF[dtype] + 2.0 ** -22) * np.abs(ref["grad"]) + LEAST[dtype]
    args = (c["z"], c["off"], c["ids"], c["q"])
    before = c["buf"].clone()
    o, d = rh.rl_distill_fwd_bwd(*args, c["dl"], p, dlogits=grad)
    f = rh.rl_distill_fwd(*args, p)
    d2, st2 = rh.rl_distill_bwd(*args, p, f.saved, c["dl"])
    assert o.status_bits() == f.status_bits() == int(st2.item()) == 0
    near(o.loss, ref["loss"], t_loss, "loss")
    near(o.mass, ref["mass"], (1.1 * eps + 2.0 ** -22) * ref["mass"] + 1e-12, "mass")
    near(d.float(), ref["grad"], t_grad, "gradient")
    near(d2.float(), ref["grad"], t_grad, "gradient of the two calls")
    assert torch.equal(f.loss, o.loss) and torch.equal(f.mass, o.mass)
    assert torch.equal(before, c["buf"])                    # the inputs stay as they are
    o3, d3 = rh.rl_distill_fwd_bwd(*args, c["dl"], p)
    assert torch.equal(o3.loss, o.loss) and torch.equal(d3, d)      # the same again
    # in place, by one call and by two
    z0 = c["z"].clone()
    z1 = c["z"]
    _, d4 = rh.rl_distill_fwd_bwd(*args, c["dl"], p, dlogits=z1)
    assert d4 is z1 and torch.equal(z1, d)
    z1.copy_(z0)
    d5, _ = rh.rl_distill_bwd(*args, p, f.saved, c["dl"], dlogits=z1)
    assert torch.equal(d5, d2)
    z1.copy_(z0)
    gap = torch.ones_like(c["buf"], dtype=torch.bool)
    gap.as_strided(c["z"].shape, c["z"].stride(), c["z"].storage_offset()).zero_()
    assert torch.equal(c["buf"][gap], before[gap])          # nothing between the rows is written
    return o, d


KINDS = [("forward", False), ("forward", True), ("reverse", True), ("jsd", True)]


@pytest.mark.parametrize("kind,tail", KINDS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 300, 1000, 5003, 32768])
def test_against_the_definition(kind, tail, dtype, V):
    rng = np.random.default_rng(V)
    k = np.minimum(rng.integers(0, 40, 9), V)
    k[0], k[-1] = min(1, V), V if V < 2000 else min(V, 700)         # one token; all of the vocabulary, or more than a block's threads
    T, beta = {1: 1.0, 7: 0.5, 300: 2.0}.get(V, 0.7), 0.3
    p = rh.DistillParams(kind=kind, tail=tail, temperature=T, beta=beta)
    check(make(9, V, dtype, k, T, tail), p, dtype)


@pytest.mark.parametrize("kind,tail", KINDS)
def test_long_supports(kind, tail):
    """Supports that do not stay in a block's registers, on rows of several blocks."""
    p = rh.DistillParams(kind=kind, tail=tail, temperature=1.0, beta=0.7)
    check(make(5, 60000, "fp32", np.array([257, 3000, 60000, 1, 20000]), 1.0, tail), p, "fp32")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 151936), (3, 50257), (40, 65537), (300, 4099)])
def test_long_and_many_rows(dtype, N, V):
    p = rh.DistillParams(kind="reverse", tail=True, temperature=1.0)
    check(make(N, V, dtype, np.arange(N) * 13 % 90, 1.0, True), p, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,pad,shift", [(1001, 0, 0), (1000, 1, 0), (1000, 3, 5), (64, 7, 1), (9, 2, 3), (5000, 8, 8), (33, 0, 1)])
def test_strides_and_alignments(dtype, V, pad, shift):
    p = rh.DistillParams(kind="jsd", tail=True, temperature=1.3, beta=0.6)
    k = np.array([3, 0, 5, min(V, 200), 1, 2])
    check(make(6, V, dtype, k, 1.3, True, pad=pad, shift=shift), p, dtype)
    # gradients with another stride and alignment than the logits
    c = make(6, V, dtype, k, 1.3, True, pad=pad, shift=shift)
    g = torch.full((6 * (V + 5) + 2,), 3.0, dtype=DT[dtype], device="cuda")
    d = g[2:].as_strided((6, V), (V + 5, 1), 2)
    check(c, p, dtype, grad=d)
    rest = torch.ones_like(g, dtype=torch.bool)
    rest.as_strided((6, V), (V + 5, 1), 2).zero_()
    assert bool((g[rest] == 3).all())


def test_the_longest_rows():
    for dtype, V in (("fp32", 450000), ("bf16", 900000)):
        p = rh.DistillParams(kind="forward", tail=True)
        check(make(2, V, dtype, np.array([5, 64]), 1.0, True), p, dtype)
    z = torch.zeros(1, 450001, device="cuda")
    c = make(1, 8, "fp32", np.array([1]))
    with pytest.raises(rh.RLHeadError):
        rh.rl_distill_fwd(z, c["off"], c["ids"], c["q"], rh.DistillParams())


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 of their buffer."""
    N, V = 2, 1000
    stride = (1 << 31) + 16
    buf = torch.empty(stride + V, dtype=torch.bfloat16, device="cuda")
    z = buf.as_strided((N, V), (stride, 1), 0)
    c = make(N, V, "bf16", np.array([4, 9]))
    z.copy_(c["z"])
    p = rh.DistillParams(kind="forward", tail=True)
    o, d = rh.rl_distill_fwd_bwd(c["z"], c["off"], c["ids"], c["q"], c["dl"], p)
    o2, d2 = rh.rl_distill_fwd_bwd(z, c["off"], c["ids"], c["q"], c["dl"], p, dlogits=z)
    assert torch.equal(o.loss, o2.loss) and torch.equal(d, d2)


@pytest.mark.parametrize("kind,tail", KINDS)
def test_masked_tokens_and_large_logits(kind, tail):
    """-inf among the rest and in the support, all of the rest masked, logits of size 1e4, a teacher that is sure."""
    V, N = 257, 8
    c = make(N, V, "fp32", np.full(N, 6), 1.0, tail, seed=4)
    z, off, ids = c["z"], c["off"].tolist(), c["ids"]
    free = [j for j in range(V) if j not in ids[off[0]:off[1]].tolist()]
    z[0, free[::2]] = float("-inf")
    S = ids[off[2]:off[3]].long()
    z[2] = torch.where(torch.isin(torch.arange(V, device="cuda"), S), z[2], torch.full_like(z[2], float("-inf")))
    z[3] *= 3000
    z[4] += 1e4
    z[5, ids[off[5]].long()] = float("-inf")                # a token of the support that the student cannot give
    c["q"][off[6]:off[7]] = torch.tensor([-40.0, -60.0, -90.0, 0.0, -70.0, -100.0])
    c["q"][off[7]] = float("-inf")                          # not of the support
    p = rh.DistillParams(kind=kind, tail=tail, beta=0.4)
    ref = reference(c, p)
    args = (z, c["off"], c["ids"], c["q"])
    o, d = rh.rl_distill_fwd_bwd(*args, c["dl"], p)
    eps = rest_error(1.0, V, 60.0)
    near(o.loss, ref["loss"], 1.1 * eps * ref["e_loss"] + 2.0 ** -23 * np.abs(ref["loss"]) + 2.0 ** -40 * 1e5 + 1e-12, "loss")
    near(d, ref["grad"], 3.3 * eps * ref["e_grad"] + 2.0 ** -21 * np.abs(ref["grad"]) + 2.0 ** -40 * 1e5, "gradient")
    assert o.status_bits() == (NONFINITE if kind == "forward" else 0)       # (row 5's loss is inf)
    assert np.isinf(ref["loss"][5]) == (kind == "forward")


def test_rows_without_a_teacher_and_without_weight():
    """No entry, entries without weight, dloss 0: zeros whatever the logits hold."""
    c = make(5, 100, "bf16", np.array([0, 3, 3, 0, 2]))
    off = c["off"].tolist()
    c["z"][0] = float("nan")
    c["z"][2, 5] = float("nan")
    c["q"][off[2]:off[3]] = float("-inf")
    c["dl"][:] = 1
    c["dl"][4] = 0
    c["z"][4, 7] = float("nan")
    p = rh.DistillParams(kind="reverse", tail=True)
    args = (c["z"], c["off"], c["ids"], c["q"])
    o, d = rh.rl_distill_fwd_bwd(*args, c["dl"], p)
    f = rh.rl_distill_fwd(*args, p)
    d2, _ = rh.rl_distill_bwd(*args, p, f.saved, c["dl"])
    for g in (d, d2):
        assert not g[[0, 2, 3, 4]].any() and bool(torch.isfinite(g[1]).all()) and bool(g[1].any())
    assert o.loss[[0, 2, 3]].tolist() == [0, 0, 0] and bool(torch.isnan(o.loss[4]))
    assert o.mass[[0, 2, 3]].tolist() == [0, 0, 0]


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["support", "rest", "last"])
def test_logits_that_are_not_numbers(value, where):
    c = make(3, 20001, "fp32", np.array([4, 4, 4]))
    at = {"support": int(c["ids"][4]), "rest": int([j for j in range(9) if j not in c["ids"][4:8].tolist()][0]), "last": 20000}[where]
    c["z"][1, at] = value
    c["dl"][:] = 1
    for kind, tail in KINDS:
        o, d = rh.rl_distill_fwd_bwd(c["z"], c["off"], c["ids"], c["q"], c["dl"], rh.DistillParams(kind=kind, tail=tail))
        assert o.status_bits() == NONFINITE
        assert not bool(torch.isfinite(o.loss[1])) and bool(torch.isfinite(o.loss[[0, 2]]).all())
        assert not bool(torch.isfinite(d[1]).all()) and bool(torch.isfinite(d[[0, 2]]).all())


def test_a_row_of_minus_inf_alone():
    c = make(3, 700, "bf16", np.array([4, 4, 4]))
    c["z"][1] = float("-inf")
    c["dl"][:] = 1
    for kind, tail in KINDS:
        p = rh.DistillParams(kind=kind, tail=tail)
        o, d = rh.rl_distill_fwd_bwd(c["z"], c["off"], c["ids"], c["q"], c["dl"], p)
        assert o.status_bits() == NONFINITE and not bool(torch.isfinite(o.loss[1]))
        assert bool(torch.isfinite(o.loss[[0, 2]]).all()) and bool(torch.isfinite(d[[0, 2]]).all())


def test_bad_rows_set_bits():
    p = rh.DistillParams(kind="reverse", tail=True)

    def run(change):
        c = make(4, 500, "fp32", np.array([5, 6, 7, 8]))
        change(c)
        args = (c["z"], c["off"], c["ids"], c["q"])
        o, d = rh.rl_distill_fwd_bwd(*args, c["dl"], p)
        f = rh.rl_distill_fwd(*args, p)
        d2, _ = rh.rl_distill_bwd(*args, p, f.saved, c["dl"])
        assert f.status_bits() == o.status_bits()
        for i in (0, 2, 3):     # the other rows are sound
            assert bool(torch.isfinite(d[i]).all()) and bool(torch.isfinite(d2[i]).all()) and bool(torch.isfinite(o.loss[i]))
        return o.status_bits(), o, d

    def put(name, i, v):
        return lambda c: c[name].__setitem__(i, v)
    assert run(lambda c: None)[0] == 0
    for v in (-1, 500, 1 << 30):
        assert run(put("ids", 7, v))[0] & ID_RANGE
    assert run(put("q", 7, float("nan")))[0] == LOGQ
    assert run(put("q", 7, float("inf")))[0] == LOGQ
    assert run(put("q", 7, 0.1))[0] == LOGQ
    assert run(lambda c: c["ids"].__setitem__(slice(6, 8), c["ids"][[7, 6]].clone()))[0] == ROW_ORDER
    assert run(lambda c: c["ids"].__setitem__(7, c["ids"][6].clone()))[0] == ROW_ORDER
    for i, v in ((1, -1), (4, 1 << 40), (2, 1)):
        bits, o, d = run(put("off", i, v))
        assert bits & OFFSETS
    # an id outside the vocabulary is left out
    _, o, d = run(put("ids", 10, 500))
    c = make(4, 500, "fp32", np.array([5, 6, 7, 8]))
    keep = torch.tensor([i for i in range(26) if i != 10], device="cuda")
    off = torch.tensor([0, 5, 10, 17, 25], device="cuda")
    o2, d2 = rh.rl_distill_fwd_bwd(c["z"], off, c["ids"][keep].contiguous(), c["q"][keep].contiguous(), c["dl"], p)
    assert torch.equal(o.loss, o2.loss) and torch.equal(d, d2)


@pytest.mark.parametrize("kind,tail", KINDS)
def test_gradient_against_differences(kind, tail):
    """Central differences of the kernel's own loss, each from two rows with one logit moved by h.  Errors: the loss's own, about
    2^-22 of its size and of the rest's terms, over h, and h^2 / 6 times a third derivative, at most 2 / T^3 here."""
    V, h, T = 24, 2.0 ** -6, 1.5
    c = make(1, V, "fp32", np.array([7]), T, tail, seed=11)
    z = c["z"][0]
    rows = z.repeat(2 * V, 1)
    rows[torch.arange(V), torch.arange(V)] += h
    rows[V + torch.arange(V), torch.arange(V)] -= h
    step = (rows[torch.arange(V), torch.arange(V)] - rows[V + torch.arange(V), torch.arange(V)]).double()
    p = rh.DistillParams(kind=kind, tail=tail, temperature=T, beta=0.35)
    n = 2 * V
    off = torch.arange(n + 1, device="cuda") * 7
    o = rh.rl_distill_fwd(rows, off, c["ids"].repeat(n), c["q"].repeat(n), p)
    got = (o.loss[:V].double() - o.loss[V:].double()) / step
    _, d = rh.rl_distill_fwd_bwd(c["z"], c["off"], c["ids"], c["q"], torch.ones(1, device="cuda"), p)
    size = float(o.loss.abs().max()) + 1
    tol = 2 * size * 2.0 ** -22 / (2 * h) + h * h / 6 * 2 / T ** 3
    assert float((got - d[0].double()).abs().max()) <= tol, float((got - d[0].double()).abs().max())


def test_graphs_streams_and_kept_outputs():
    """Captured with changing inputs, and on two streams at once."""
    c = make(64, 32768, "bf16", np.arange(64) % 30)
    p = rh.DistillParams(kind="jsd", tail=True, beta=0.5)
    args = (c["z"], c["off"], c["ids"], c["q"], c["dl"], p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, d = rh.rl_distill_fwd_bwd(*args, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rh.rl_distill_fwd_bwd(*args, out=o, dlogits=d)
    c["z"].copy_(c["z"].flip(0))
    c["dl"].mul_(0.5)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want, wd = rh.rl_distill_fwd_bwd(*args)
    assert torch.equal(o.loss, want.loss) and torch.equal(d, wd)
    t = torch.cuda.Stream()
    t.wait_stream(torch.cuda.current_stream())
    res = [rh.rl_distill_fwd_bwd(*args, stream=x) for x in (s, t) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a.loss, want.loss) and torch.equal(b, wd) for a, b in res)


def test_waits_that_run_out():
    """With the shortest limit a call ends, with TIMEOUT and no other bit if a wait ran out, and the next one, with the usual
    limit, is right."""
    c = make(304, 65537, "fp32", np.arange(304) % 30)
    args = (c["z"], c["off"], c["ids"], c["q"], c["dl"], rh.DistillParams(kind="reverse", tail=True))
    want, wd = rh.rl_distill_fwd_bwd(*args)
    rh.rl_set_option(rh.RL_OPT_WAIT_LIMIT_US, 1)
    try:
        bits = [rh.rl_distill_fwd_bwd(*args)[0].status_bits() for _ in range(3)]
    finally:
        rh.rl_set_option(rh.RL_OPT_WAIT_LIMIT_US, 1_000_000)
    print("bits", bits)
    assert all(b in (0, 0x200) for b in bits)
    again, d = rh.rl_distill_fwd_bwd(*args)
    assert again.status_bits() == 0 and torch.equal(again.loss, want.loss) and torch.equal(d, wd)


def test_no_rows():
    z = torch.zeros(0, 100, device="cuda")
    e = torch.zeros(0, device="cuda")
    o, d = rh.rl_distill_fwd_bwd(z, torch.zeros(1, dtype=torch.int64, device="cuda"), e.to(torch.int32), e, e, rh.DistillParams())
    assert o.loss.numel() == 0 and d.shape == z.shape and o.status_bits() == 0
