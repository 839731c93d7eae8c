"""Verification at the ends of the range: small temperatures, masks of finite size."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh  # noqa: F401
from test_gpu_verify import DT, Half, call, check

pytestmark = pytest.mark.gpu


def rows_case(z, zd, temp, temp_d, seed, likely=0.6):
    """Requests of three rows; candidates are the largest logits of either side or a token whose p or q does not underflow in the
    64-bit reference (u q < p of two numbers below that is not its to decide)."""
    rng = np.random.default_rng(seed)
    T, V = z.shape
    step = np.zeros(T, int)
    for t in range(T):
        a, b = ((x[t].double() - x[t].double().max()) / float(k[t]) for x, k in ((z, temp), (zd, temp_d)))
        some = torch.nonzero(torch.maximum(a, b) > -700)[:, 0]
        x = rng.random()
        step[(t + 1) % T] = int(a.argmax() if x < likely else b.argmax() if x < likely + 0.15 else some[rng.integers(0, len(some))])
    f = lambda k: (rng.integers(0, 1 << 24, k) / 2.0 ** 24).astype(np.float32)  # noqa: E731
    return dict(step=step, cu=np.arange(0, T + 1, 3), u=f(T), un=f(T // 3), V=V, ctx=np.zeros(T // 3, int), target=Half(V, z, temp),
                draft=Half(V, zd, temp_d))


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
@pytest.mark.parametrize("T", [1e-5, 3e-7, 3e-8, 1e-8, 3e-9, 1e-9, 1e-10, 1e-12, 1e-20, 1e-33])
def test_small_temperatures(T, dtype):
    """Exponents z / T of any size, on either side and on both, over several chunks: rows whose largest logits are apart."""
    n, V = 24, 4500
    g = torch.Generator().manual_seed(int(-np.log10(T) * 10))
    z = (torch.randn(n, V, generator=g) * 6).to(DT[dtype])
    zd = (z.float() + torch.randn(n, V, generator=g)).to(DT[dtype])
    for x in (z, zd):           # (no ties)
        x[torch.arange(n), torch.randint(0, V, (n,), generator=g)] = 40.0
    small, one = np.full(n, T, np.float32), np.ones(n, np.float32)
    for a, b in ((small, small), (small, one), (one, small)):
        check(rows_case(z, zd, a, b, 5))
        check(dict(rows_case(z, zd, a, b, 6), draft=None))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("mask", [-6e4, -1e9, -1e10, -1e20, None])
@pytest.mark.parametrize("T", [1.0, 0.3, 0.1])
def test_whole_chunks_masked_by_a_finite_number(T, mask, dtype):
    """Masks of a size between the logits' own and the type's lowest, over more than a chunk's tokens of either side."""
    least = torch.finfo(DT[dtype]).min
    mask = least if mask is None else max(mask, least)
    n, V = 24, 9000
    g = torch.Generator().manual_seed(3)
    z = (torch.randn(n, V, generator=g) * 3).to(DT[dtype])
    zd = (z.float() + 0.7 * torch.randn(n, V, generator=g)).to(DT[dtype])
    z[:, 2000:6500] = mask
    z[1::4, :8990] = mask       # all but a few
    zd[::2, 2040:6400] = mask
    zd[1::2, 4000:] = mask
    t = np.full(n, T, np.float32)
    check(rows_case(z, zd, t, t, 7))
    check(dict(rows_case(z, zd, t, t, 8), draft=None))
    ids = [np.array([1, 7, 4000, 5000, 8995])] * n
    lq = [np.log(np.array([0.1, 0.2, 0.3, 0.3, 0.1])).astype(np.float32)] * n
    c = rows_case(z, zd, t, t, 9, likely=1.0)       # (a support row gives a token without an entry no probability at all)
    c["step"][1::3] = 7
    check(dict(c, draft=Half(V, ids=ids, lq=lq)))


SPACING = [0.9, 1.6, 5, 15, 40, 90, 110, 123, 125, 126.5, 127.2, 127.5, 127.9, 128.5, 200]


@pytest.mark.parametrize("M", [20.0, 3.0])
@pytest.mark.parametrize("steps", SPACING)
def test_temperatures_at_which_one_float_is_many_powers_of_two(steps, M):
    """T such that two floats next to each other near the largest logit have weights 2^-steps apart; a float below the largest on
    either side, twice and in every part."""
    n, V = 24, 700
    T = np.float32(np.log2(np.e) * float(np.spacing(np.float32(M))) / steps)
    rng = np.random.default_rng(int(steps * 10))
    z, zd = torch.full((n, V), -5.0), torch.full((n, V), -5.0)
    for t in range(n):
        for x in (z, zd):
            x[t, 50::90] = float(np.nextafter(np.float32(M), np.float32(0)))
            x[t, 51::90] = float(np.nextafter(np.nextafter(np.float32(M), np.float32(0)), np.float32(0)))
            x[t, rng.integers(0, V)] = M
    small, one = np.full(n, T, np.float32), np.ones(n, np.float32)
    for a, b in ((small, small), (small, one), (one, small)):
        check(rows_case(z, zd, a, b, 5), skips=4)
        check(dict(rows_case(z, zd, a, b, 6), draft=None), skips=4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("steps", SPACING)
def test_ties_beside_a_sure_draft_at_small_temperatures(steps, dtype):
    """The target's largest logit many times, the draft's once among them: the token is not the draft's, and those after it
    in its part of the row are where they belong."""
    R, V, ties = 32, 1500, 1024
    T = np.float32(np.log2(np.e) * float(np.spacing(np.float32(20.0))) / steps)
    z, zd = torch.full((2 * R, V), -5.0), torch.full((2 * R, V), -5.0)
    z[:, :ties] = 20.0
    step, un = np.zeros(2 * R, int), np.zeros(R, np.float32)
    for r in range(R):
        x = 128 * (r % 8) + 5 + r
        zd[2 * r, x] = 20.0
        step[2 * r + 1] = x
        un[r] = (128 * (r % 8) + 60.3 + r) / (ties - 1)
    small = np.full(2 * R, T, np.float32)
    c = dict(step=step, cu=np.arange(0, 2 * R + 1, 2), u=np.full(2 * R, 0.5, np.float32), un=un, V=V, ctx=np.zeros(R, int),
             target=Half(V, z.to(DT[dtype]), small), draft=Half(V, zd.to(DT[dtype]), small))
    check(c)
    check(dict(c, draft=Half(V, zd.to(DT[dtype]), np.ones(2 * R, np.float32))))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [3.0, 1.0, 0.7, 0.1, 1e-6])
def test_support_rows_beside_drafts_masked_by_the_lowest_number(T, dtype):
    """Tokens of the target's support row whose draft logits are the type's lowest number have no probability in the draft, whatever
    the temperature makes of the number: all of the target's is left."""
    R, V = 32, 3000
    g = torch.Generator().manual_seed(4)
    zd = (torch.randn(2 * R, V, generator=g) * 3).to(DT[dtype])
    ids = [np.array([1, 7, 700, 1500, 2995])] * (2 * R)
    lq = [np.log(np.array([0.1, 0.2, 0.3, 0.3, 0.1])).astype(np.float32)] * (2 * R)
    step = np.zeros(2 * R, int)
    for r in range(R):
        zd[2 * r, [1, 700, 2995]] = torch.finfo(DT[dtype]).min
        zd[2 * r, 7] = 400.0                # what the draft gives, more often than the target
        step[2 * r + 1] = 7
    un = ((np.arange(R) + 0.5) / R).astype(np.float32)
    temp = np.full(2 * R, T, np.float32)
    c = dict(step=step, cu=np.arange(0, 2 * R + 1, 2), u=np.full(2 * R, 0.9, np.float32), un=un, V=V, ctx=np.zeros(R, int),
             target=Half(V, ids=ids, lq=lq), draft=Half(V, zd, temp))
    ref, _ = check(c)
    assert set(ref["tokens"][::2]) == {1, 700, 1500, 2995}


def test_logits_of_no_rows():
    """A step without tokens, a step without drafts, and a row map into no rows at all."""
    V, R = 300, 3
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    none = torch.zeros(0, V, device="cuda")
    z = torch.randn(R, V, generator=torch.Generator().manual_seed(1)).cuda()
    for draft in (rh.Dist(logits=none), None):
        o = rh.rl_verify(i(), i(0, 0, 0, 0), f(), f(0.1, 0.2, 0.3), rh.Dist(logits=none), draft, vocab=V, ctx_lens=i(4, 5, 6))
        assert o.accepted.tolist() == [0, 0, 0] and o.keep_lens.tolist() == [4, 5, 6] and o.status_bits() == 0
        o = rh.rl_verify(i(), i(0), f(), f(), rh.Dist(logits=none), draft, vocab=V)
        assert o.status_bits() == 0
    # requests of one token: a draft of no rows is not looked at
    rows = rh.Dist(logits=none, rows=i(0, 0, 0))
    args = (i(1, 2, 3), i(0, 1, 2, 3), f(0, 0, 0), f(0.1, 0.5, 0.9), rh.Dist(logits=z))
    o, want = rh.rl_verify(*args, rows, vocab=V), rh.rl_verify(*args, None, vocab=V)
    assert torch.equal(o.tokens, want.tokens) and torch.equal(o.logq, want.logq) and o.status_bits() == 0
    # a candidate whose draft row does not exist: not a sure draft
    args = (i(1, 2, 3), i(0, 3), f(0.5, 0.5, 0.5), f(0.5), rh.Dist(logits=z))
    assert rh.rl_verify(*args, rows, vocab=V).status_bits() == 0x21          # OFFSETS, EMPTY_ROW
    assert rh.rl_verify(*args, None, vocab=V).status_bits() == 0


@pytest.mark.parametrize("form", ["dense", "rows", "sure"])
@pytest.mark.parametrize("V", [2, 130, 1500])
def test_nothing_left_but_the_sums_own_error(V, form):
    """Both sides give one token all but e^-40; a candidate that only the draft gives anything (e^-46) is turned down.  What is left
    of the likely token, 1e-20, is far below the sums' accuracy, and of the others it is less by 1e6 and more: the token is the likely
    one, not any that happens to lie beside it."""
    R = 128
    rng = np.random.default_rng(V)
    T, Td = rng.uniform(0.01, 0.05, 2 * R), rng.uniform(0.001, 0.05, 2 * R)
    M, Md = rng.uniform(3, 9, 2 * R), rng.uniform(3, 9, 2 * R)
    z = torch.from_numpy(M[:, None] - 200 * T[:, None] * np.ones(V)).float()
    zd = torch.from_numpy(Md[:, None] - 200 * Td[:, None] * np.ones(V)).float()
    a = rng.integers(0, V, 2 * R)
    step = np.zeros(2 * R, int)
    rows = torch.arange(2 * R)
    z[rows, a], zd[rows, a] = torch.from_numpy(M).float(), torch.from_numpy(Md).float()
    b = (a + 1 + rng.integers(0, max(V - 1, 1), 2 * R) % (V - 1)) % V
    step[1::2] = b[::2]
    zd[rows, b] = torch.from_numpy(Md - 46 * Td).float()
    temp, temp_d = T.astype(np.float32), Td.astype(np.float32)
    draft = Half(V, zd, temp_d) if form == "dense" else None
    if form == "rows":
        ids = [np.sort([x, y]) for x, y in zip(a, b)]
        draft = Half(V, ids=ids, lq=[np.where(i == x, 0, -46).astype(np.float32) for i, x in zip(ids, a)])
    c = dict(step=step, cu=np.arange(0, 2 * R + 1, 2), u=np.full(2 * R, 0.9, np.float32), un=rng.random(R).astype(np.float32), V=V,
             ctx=np.zeros(R, int), target=Half(V, z, temp), draft=draft)
    for dtype in ("fp32", "bf16"):
        o = call(dict(c, target=Half(V, z.to(DT[dtype]), temp)))
        assert not o.accepted.any() and o.status_bits() == 0
        assert (o.tokens.cpu().numpy()[::2] == a[::2]).all(), np.flatnonzero(o.tokens.cpu().numpy()[::2] != a[::2])
