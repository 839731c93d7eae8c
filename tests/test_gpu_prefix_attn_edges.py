"""rl_prefix_attn where its kernels differ from one another or meet what they may not follow.

The bars are those of test_gpu_prefix_attn.py.
"""
import pytest
import torch

import lm_head_gb300 as rh
from test_gpu_prefix_attn import BF, HF, LENGTHS, Case

pytestmark = pytest.mark.gpu

# a step whose rows are done by tiles of 16, by one tile of up to 128 rows, and by two such tiles
KINDS = [("warp", dict(groups=[3], prefixes=[70], q_lens=[1] * 3, kv_lens=[1, 17, 64])),
         ("warp, one part", dict(groups=[], prefixes=[], q_lens=[1, 3], kv_lens=[200, 40])),
         ("keys", dict(groups=[17], prefixes=[300], q_lens=[1] * 17, kv_lens=[1 + 9 * i for i in range(17)])),
         ("keys, one part", dict(groups=[], prefixes=[], q_lens=[20, 11], kv_lens=[150, 11])),
         ("rows", dict(groups=[2], prefixes=[131], q_lens=[130, 70], kv_lens=[130, 400])),
         ("rows, one part", dict(groups=[], prefixes=[], q_lens=[140], kv_lens=[190]))]


def make(kind, D=64, page=16, dtype=BF, seed=1):
    return Case(Hq=8, Hkv=2, D=D, page=page, dtype=dtype, seed=seed, **dict(KINDS)[kind])


@pytest.mark.parametrize("kind", [k for k, _ in KINDS])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF)])
def test_scale_zero_is_the_mean_of_the_values(kind, D, dtype):
    c = make(kind, D, dtype=dtype)
    c.scale = 0.0
    c.check()


@pytest.mark.parametrize("kind", [k for k, _ in KINDS])
def test_a_nan_query_gives_a_nan_row(kind):
    """One row of one head is NaN in output and lse; all others are what they are without it."""
    c = make(kind)
    want = c.check()
    for t in {0, c.q.shape[0] - 1}:
        q = c.q.clone()
        q[t, 3, 5] = float("nan")
        a = c.run(q)
        assert bool(torch.isnan(a.out[t, 3]).all()) and bool(torch.isnan(a.lse[t, 3]))
        rest = torch.ones(c.q.shape[:2], dtype=torch.bool, device="cuda")
        rest[t, 3] = False
        assert torch.equal(a.out[rest], want.out[rest]) and torch.equal(a.lse[rest], want.lse[rest])


def put(c, r, key, k=None, v=None):
    """Overwrites key `key` of own pages r, or of group r - len(q_lens)'s prefix, in the cache."""
    R = len(c.q_lens)
    table = c.table[r] if r < R else c.ptable[r - R]
    page = c.kc.shape[2]
    for cache, x in ((c.kc, k), (c.vc, v)):
        if x is not None:
            cache[int(table[key // page]), :, key % page] = x


@pytest.mark.parametrize("kind", [k for k, _ in KINDS])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_nan_key_or_value_reaches_every_row_that_sees_it(kind, what):
    c = make(kind)
    want = c.check()
    R = len(c.q_lens)
    first = [sum(c.q_lens[:r]) for r in range(R + 1)]
    for r, key in [(R - 1, 0)] + ([(R, len(c.keys[R][0]) // 2)] if c.groups else []):
        kc, vc = c.kc.clone(), c.vc.clone()
        put(c, r, key, **{what: float("nan")})
        a = c.run()
        hit = torch.zeros(c.q.shape[0], dtype=torch.bool, device="cuda")
        hit[first[R - 1] if r == R - 1 else 0:] = True       # key 0 is seen by all of the last request's tokens
        assert bool(torch.isnan(a.out[hit]).all())
        if what == "k":
            assert bool(torch.isnan(a.lse[hit]).all())
        assert torch.equal(a.out[~hit], want.out[~hit]) and torch.equal(a.lse[~hit], want.lse[~hit])
        c.kc, c.vc = kc, vc


@pytest.mark.parametrize("kind", [k for k, _ in KINDS])
def test_infinite_scores(kind):
    """A key with an infinity: a row whose score it makes +inf is NaN, as in softmax; where it makes it
    -inf the key has no weight (and a row of no other key is one that sees none)."""
    c = make(kind)
    r = len(c.q_lens) - 1
    x = c.keys[r][0][0].clone()
    x[:, 7] = float("inf")
    put(c, r, 0, k=x.cuda())
    c.keys[r] = (torch.cat([x[None], c.keys[r][0][1:]]), c.keys[r][1])
    a = c.run()
    out, lse, vmax = c.reference()
    out[lse == -float("inf")] = 0
    bad = torch.isnan(out).any(-1)
    assert bool(bad.any()) and bool((~bad).any())
    got = a.out.cpu().double()
    assert torch.equal(torch.isnan(got).any(-1), bad)
    eps = torch.finfo(c.q.dtype).eps
    bar = eps / 2 * (out.abs() + vmax[..., None]) + 2.0 ** -16 * vmax[..., None]
    assert bool(((got - out).abs() <= bar)[~bad].all())


@pytest.mark.parametrize("kind", ["keys", "rows"])
@pytest.mark.parametrize("groups", [[], [3, 5]])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
def test_a_wait_that_runs_out_ends_the_tensor_core_kernels(kind, groups, D, dtype):
    """With a limit of 1 us waits run out for certain (a step of these kernels takes longer): the call
    ends with TIMEOUT and no other bit, and the next one, with the usual limit, is right."""
    n = 32 if kind == "keys" else 100
    c = Case(groups, [700] * len(groups), [n] * 8, [5000 - 300 * i for i in range(8)], 8, 2, D, 16, dtype, 10)
    want = c.run()
    rh.rl_set_option(rh.RL_OPT_WAIT_LIMIT_US, 1)
    try:
        bits = [c.run().status_bits() for _ in range(3)]
    finally:
        rh.rl_set_option(rh.RL_OPT_WAIT_LIMIT_US, 1_000_000)
    assert bits == [0x200] * 3
    again = c.run()
    assert again.status_bits() == 0 and torch.equal(again.out, want.out) and torch.equal(again.lse, want.lse)


def test_a_prefix_without_its_bound_is_not_lost():
    """max_prefix left out is the table's width; a bound of 0 with a prompt is an error, not a step
    without its prompt."""
    for kind in ("warp", "keys", "rows"):
        c = make(kind)
        c.check()
        a = rh.rl_prefix_attn(c.q, c.kc, c.vc, c.cu, c.kvt, c.table, max_q=c.bounds["max_q"], max_kv=c.bounds["max_kv"],
                              group_offsets=c.go, prefix_lens=c.pl, prefix_table=c.ptable, scale=c.scale)
        c.check(a)
        assert c.run(max_prefix=0).status_bits() == LENGTHS
        c.pl = torch.zeros_like(c.pl)
        assert c.run(max_prefix=0).status_bits() == 0
        c.pl = torch.full_like(c.pl, -3)
        assert c.run(max_prefix=0).status_bits() == LENGTHS


# all of a step's rows over prefix and own keys in one block: many tokens a request, no join
BOTH = dict(groups=[2, 0, 3, 1], prefixes=[300, 50, 129, 1], q_lens=[33, 257, 1, 0, 300, 128, 400, 129],
            kv_lens=[33, 266, 6, 0, 427, 192, 600, 130], stray=1)


@pytest.mark.parametrize("kind", ["warp", "keys", "rows", "both"])
def test_group_offsets_that_do_not_add_up_set_status(kind):
    if kind == "both":
        c = Case(Hq=16, Hkv=2, D=64, page=16, dtype=BF, seed=2, **BOTH)
        assert c.run().ws.numel() == 1          # no parts to join
    else:
        c = make(kind)
    R, G = len(c.q_lens), len(c.groups)
    for bad in (R + 1, -1):
        go = c.go.clone()
        go[-1 if bad > 0 else 0] = bad
        good, c.go = c.go, go
        assert c.run().status_bits() == LENGTHS
        c.go = good
    if G > 1:
        c.go = c.go.flip(0).contiguous()
        assert c.run().status_bits() == LENGTHS


@pytest.mark.parametrize("Hq", [1, 8])
def test_strides_of_axes_of_one_entry_mean_nothing(Hq):
    """One token, or one head, whose unused stride is odd."""
    c = Case([1], [40], [1], [20], Hq, 1, 64, 16, BF, 3)
    want = c.check()
    a = c.run(torch.as_strided(c.q, c.q.shape, (515, c.q.stride(1), 1)))
    assert torch.equal(a.out, want.out) and torch.equal(a.lse, want.lse)
    if Hq == 1:
        c = Case([1], [40], [5], [20], 1, 1, 64, 16, BF, 3)
        want = c.check()
        a = c.run(torch.as_strided(c.q, c.q.shape, (c.q.stride(0), 3, 1)))
        assert torch.equal(a.out, want.out) and torch.equal(a.lse, want.lse)
