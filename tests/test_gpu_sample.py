"""rl_sample against its definition in 64 bits.

Tokens, support sets and counts are equal to the reference's in every row whose random numbers
and set border keep 1e-9 of the total away from a border of the cumulative weights (the sums
carry 2^-37 = 7e-12 of the largest weight and term, so 1e-9 leaves two orders); the inputs here
have such a margin in nearly every row, and each test asserts that.  Log-probabilities are the
fp32 rounding (2^-24 relative) of a float-pair sum: 2^-23 relative, plus 1e-9 for the ln of the
sum, is the bar.
"""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from generation_ref import sample_reference

pytestmark = pytest.mark.gpu
EMPTY_ROW, NONFINITE, KNOB, CAPACITY = 0x20, 0x100, 0x2000, 0x4000
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def run(z, u, capacity=None, **kn):
    """z: device logits; kn: numpy knobs or None."""
    c = lambda a, dt: None if a is None else torch.tensor(np.asarray(a), dtype=dt, device="cuda")  # noqa: E731
    cap = z.numel() + z.shape[0] * u.shape[1] if capacity is None else capacity
    o = rh.rl_sample(z, c(u, torch.float32), temperature=c(kn.get("temperature"), torch.float32),
                     top_k=c(kn.get("top_k"), torch.int32), top_p=c(kn.get("top_p"), torch.float32),
                     min_p=c(kn.get("min_p"), torch.float32), capacity=cap)
    torch.cuda.synchronize()
    return o


def f32(a):
    return None if a is None else np.asarray(a, np.float32).astype(np.float64)


def check(z, u, bits=0, rows=None, **kn):
    o = run(z, u, **kn)
    ref = sample_reference(z.double().cpu().numpy(), f32(u), f32(kn.get("temperature")), kn.get("top_k"),
                           f32(kn.get("top_p")), f32(kn.get("min_p")))
    N = z.shape[0]
    sure = ref["margin"] > 1e-9
    assert sure.mean() > 0.9
    tok, lq, off = o.tokens.cpu().numpy(), o.logq.cpu().double().numpy(), o.offsets.cpu().numpy()
    ids, slq = o.ids.cpu().numpy(), o.support_logq.cpu().double().numpy()
    np.testing.assert_array_equal(tok[sure], ref["tokens"][sure])
    ok = np.isfinite(ref["logq"]) & sure[:, None]
    assert np.all(np.abs(lq[ok] - ref["logq"][ok]) <= 2.0 ** -23 * np.abs(ref["logq"][ok]) + 1e-9)
    assert np.all(lq[~np.isfinite(ref["logq"])] == -np.inf)
    np.testing.assert_array_equal(o.replayed.cpu().numpy(), ref["replayed"])
    assert off[0] == 0
    for r in range(N):
        if not sure[r]:
            continue
        a, b = off[r], off[r + 1]
        np.testing.assert_array_equal(ids[a:b], ref["ids"][r], err_msg=f"row {r}")
        e = ref["support_logq"][r]
        assert np.all(np.abs(slq[a:b] - e) <= 2.0 ** -23 * np.abs(e) + 1e-9), r
    assert o.status_bits() == bits, (rh.status_names(o.status_bits()), rh.status_names(bits))
    return o, ref


def logits(N, V, dt, seed, spread=2.5, likely=8):
    g = torch.Generator().manual_seed(seed)
    z = spread * torch.randn(N, V, generator=g)
    if V > 2 * likely:
        z.scatter_(1, torch.randint(0, V, (N, likely), generator=g), 7 + 5 * torch.rand(N, likely, generator=g))
    return z.to(DT[dt]).cuda()


def rand_u(N, K, seed):
    return (np.random.RandomState(seed).randint(0, 1 << 24, (N, K)) + 0.5) / (1 << 24) * (1 - 2.0 ** -23)


def knobs(kind, N, V, seed):
    r = np.random.RandomState(seed)
    kn = {}
    if kind in ("all", "mixed"):
        kn["temperature"] = r.uniform(0.3, 1.5, N)
    if kind in ("top_k", "all", "mixed", "k_p"):
        kn["top_k"] = r.randint(1, max(2, min(V, 300)), N)
    if kind in ("top_p", "all", "mixed", "k_p", "p_min"):
        kn["top_p"] = r.uniform(0.3, 0.99, N)
    if kind in ("min_p", "all", "mixed", "p_min"):
        kn["min_p"] = r.uniform(0.001, 0.3, N)
    if kind == "mixed":
        kn["top_k"][::2] = 0
        kn["top_p"][::3] = 1.0
        kn["min_p"][::5] = 0.0
        kn["temperature"][::7] = 0.0
        for k in ("top_k", "top_p", "min_p"):
            kn[k][1::11] = {"top_k": V + 3, "top_p": 1.5, "min_p": -1.0}[k]
    return kn


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p", "min_p", "k_p", "p_min", "all", "mixed"])
@pytest.mark.parametrize("N,V,K", [(3, 1000, 1), (17, 4099, 5), (5, 50257, 17)])
def test_matches_the_definition(N, V, K, kind, dt):
    check(logits(N, V, dt, V + N), rand_u(N, K, N), **knobs(kind, N, V, 7 * N + K))


@pytest.mark.parametrize("V", [1, 2, 3, 31, 127, 128, 129, 1023, 1024, 1025, 2047, 8192])
def test_odd_vocabularies(V):
    N = 9
    for kind in ("none", "mixed", "top_p"):
        check(logits(N, V, "fp32", V), rand_u(N, 3, V), **knobs(kind, N, V, V))


def test_the_heads_vocabulary_broad_and_narrow_rows():
    """151,936 logits: nuclei from one token to most of the vocabulary."""
    V = 151936
    z = torch.cat([logits(4, V, "fp32", 1, spread=s) for s in (0.2, 1.0, 2.0, 3.5)])
    N = z.shape[0]
    for kn in ({}, {"top_p": np.full(N, 0.97)}, {"top_p": np.full(N, 0.5)}, {"min_p": np.full(N, 1e-4)},
               {"top_k": np.full(N, 60000)}, {"top_k": np.full(N, 3000), "top_p": np.full(N, 0.9)},
               {"top_p": np.full(N, 0.9), "min_p": np.full(N, 1e-5)}):
        check(z, rand_u(N, 4, 3), **kn)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_ties_keep_the_lowest_indices(dt):
    """Few distinct values: borders fall among equal logits, more than any list holds."""
    N, V = 6, 30011
    g = torch.Generator().manual_seed(5)
    z = torch.randint(0, 4, (N, V), generator=g).to(DT[dt]).cuda()
    z[2] = 1.25                       # all equal
    z[3, 1:] = -3.0                   # one above the rest
    for kn in ({"top_k": [1, 100, 17, 2, 20000, 29999]}, {"top_p": [0.1, 0.5, 0.37, 0.9, 0.999, 0.7]},
               {"top_k": [9000, 12000, 29000, 7, 5, 30010], "top_p": [0.5, 0.9, 0.25, 0.99, 0.4, 0.6]},
               {"min_p": np.full(N, 0.3), "top_p": np.full(N, 0.45)}, {"temperature": np.zeros(N)}):
        check(z, rand_u(N, 3, 11), **kn)


def test_masked_logits():
    """-inf and the type's lowest value as masks; a row of lowest values; a row with one token left;
    a row with none; NaN and +inf."""
    N, V = 8, 2000
    z = logits(N, V, "fp32", 3)
    low = torch.finfo(torch.float32).min
    z[0, ::2] = float("-inf")
    z[1, ::2] = low
    z[2] = low
    z[3] = float("-inf")
    z[3, 777] = 0.5
    z[5, 100:] = low
    for kind in ("none", "top_k", "top_p", "min_p", "all"):
        check(z, rand_u(N, 4, 9), **knobs(kind, N, V, 1))
    z[6] = float("-inf")
    z[4, 5], z[4, 6], z[7, 0] = float("nan"), float("inf"), float("-inf")
    for kind in ("none", "all"):
        check(z, rand_u(N, 4, 9), bits=EMPTY_ROW | NONFINITE, **knobs(kind, N, V, 1))


def test_extreme_temperatures_and_large_logits():
    N, V = 6, 5000
    z = logits(N, V, "fp32", 8) * torch.tensor([1.0, 100.0, 1000.0, 1e-3, 30.0, 1.0], device="cuda")[:, None]
    T = np.array([1e-3, 1.0, 50.0, 1e-4, 0.01, 1e6])
    for kn in ({}, {"top_k": np.full(N, 40)}, {"top_p": np.full(N, 0.9)}, {"min_p": np.full(N, 0.01)}):
        check(z, rand_u(N, 5, 2), temperature=T, **kn)


def test_knobs_out_of_range():
    N, V = 6, 500
    z = logits(N, V, "bf16", 4)
    check(z, rand_u(N, 2, 1), bits=KNOB, temperature=[-1.0, np.nan, np.inf, 1.0, 1.0, 0.5])
    check(z, rand_u(N, 2, 1), bits=KNOB, top_p=[np.nan, 0.5, 0.0, -3.0, 1.0, 2.0], min_p=[0, np.nan, 5.0, 0.1, -1, 1.0])
    o = run(z, np.array([[1.0], [-0.5], [np.nan], [0.0], [0.5], [0.999999]]))
    assert o.status_bits() == KNOB and bool(((o.tokens >= 0) & (o.tokens < V)).all())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_strided_and_unaligned_rows(dt):
    N, V = 5, 3001
    buf = logits(N, V + 7, dt, 6)
    for z in (buf[:, 1:V + 1], buf[:, 4:V + 4], buf[1:2, 3:V + 3]):
        for kind in ("none", "all"):
            check(z, rand_u(z.shape[0], 3, 2), **knobs(kind, z.shape[0], V, 3))


def test_the_largest_vocabulary():
    V = 1 << 20
    z = logits(3, V, "bf16", 21)
    for kn in ({}, {"top_k": [7, 100000, 0], "top_p": [0.9, 0.5, 0.97]}):
        check(z, rand_u(3, 3, 6), **kn)


def test_capacity_is_respected():
    N, V = 5, 4000
    z, kn = logits(N, V, "fp32", 2), dict(top_p=np.full(5, 0.9))
    full = run(z, rand_u(N, 1, 1), **kn)
    nnz = full.nnz()
    cap = nnz - 3
    ids = torch.full((nnz + 8,), -7, dtype=torch.int32, device="cuda")
    o = rh.rl_sample(z, torch.tensor(rand_u(N, 1, 1), dtype=torch.float32, device="cuda"),
                     top_p=torch.full((N,), 0.9, device="cuda"), capacity=cap,
                     out=rh.SampleOut(full.tokens, full.logq, full.offsets.clone(), ids[:cap],
                                      torch.zeros(cap, device="cuda"), full.replayed, full.ws, torch.zeros_like(full.status)))
    torch.cuda.synchronize()
    assert o.status_bits() == CAPACITY and o.nnz() == nnz
    assert torch.equal(ids[:cap], full.ids[:cap]) and bool((ids[cap:] == -7).all())


def test_without_support_and_without_logq():
    N, V = 4, 3000
    z, u = logits(N, V, "fp32", 2), rand_u(N, 2, 1)
    a = run(z, u, top_k=np.full(N, 20))
    b = run(z, u, capacity=0, top_k=np.full(N, 20))
    assert b.offsets is None and torch.equal(a.tokens, b.tokens) and torch.equal(a.logq, b.logq)
    assert rh.rl_sample(z[:0], torch.zeros(0, 1, device="cuda"), capacity=5).nnz() == 0


def test_repeated_calls_are_bitwise_equal_and_a_graph_replays():
    N, V = 40, 151936
    z = logits(N, V, "bf16", 12)
    kn = knobs("mixed", N, V, 4)
    kn["top_p"][:] = 0.95
    u = rand_u(N, 9, 5)
    a, b = run(z, u, **kn), run(z, u, **kn)
    for x, y in ((a.tokens, b.tokens), (a.logq, b.logq), (a.offsets, b.offsets), (a.ids, b.ids), (a.support_logq, b.support_logq)):
        assert torch.equal(x, y)
    c = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in kn.items()}
    ut = torch.tensor(u, dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o = rh.rl_sample(z, ut, capacity=a.ids.numel(), **c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rh.rl_sample(z, ut, capacity=a.ids.numel(), out=o, **c)
    z.copy_(logits(N, V, "bf16", 13))
    g.replay()
    torch.cuda.synchronize()
    d = run(z, u, **kn)
    assert torch.equal(o.tokens, d.tokens) and torch.equal(o.offsets, d.offsets) and torch.equal(o.logq, d.logq)


def test_the_support_feeds_the_head():
    """Rows sampled here are valid evidence for the head: rl_validate_support sets no bit (masses
    within 1e-3, labels present, ascending ids), with cut and whole rows in one batch."""
    N, V, H = 64, 4096, 128
    g = torch.Generator().manual_seed(1)
    X = torch.randn(N, H, generator=g).bfloat16().cuda()
    W = (torch.randn(V, H, generator=g) * 0.2).bfloat16().cuda()
    z = (X.float() @ W.float().T).contiguous()
    kn = dict(top_p=np.where(np.arange(N) % 2 == 0, 0.97, 1.0))
    o = run(z, rand_u(N, 17, 3), **kn)
    n = o.nnz()
    batch = rh.HeadBatch(X, W, o.tokens[:, 0].contiguous(), o.logq[:, 0].contiguous(), torch.ones(N, device="cuda"),
                         o.offsets, o.ids[:n], o.support_logq[:n], o.replayed)
    assert int(rh.rl_validate_support(batch).item()) == 0
    fwd = rh.rl_head_loss_fwd(batch, rh.HeadParams())
    assert fwd.status_bits() == 0 and bool(torch.isfinite(fwd.loss).all())
