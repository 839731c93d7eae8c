"""rl_sample where its sums are longest: rows of up to 2^20 logits whose weights are all alike, and
rows in which a few likely tokens stand over a flat tail that decides the border or the draw.

The definition is evaluated in extended precision (the tail's sums lose too much in 64 bits: 150,000
equal terms next to a sum near 1).  Sums carry 2^-36 of the total: rows whose border or random
number lies nearer than 2^-35 of the total to a border of the cumulative weights may take the neighbour, and
the inputs are chosen so that none does.
"""
import math

import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from test_gpu_sample import check, run

pytestmark = pytest.mark.gpu


def f32(x):
    return float(np.float32(x))


def extended(z, u, T=1.0, p=1.0):
    """Tokens and kept ids of one row, and how far the border and the draws are from the next one."""
    x = (np.asarray(z, np.float64).astype(np.longdouble) - np.longdouble(max(z))) / np.longdouble(T)
    w = np.exp(x)
    S = np.arange(len(z))
    margin = math.inf
    if p < 1:
        order = np.lexsort((S, -x))
        c = np.cumsum(w[order])
        S = np.sort(order[:1 + int(np.count_nonzero(c[:-1] < np.longdouble(p) * c[-1]))])
        margin = float(np.min(np.abs(c - np.longdouble(p) * c[-1])) / c[-1])
    c = np.cumsum(w[S])
    at = [np.longdouble(v) * c[-1] for v in u]
    margin = min(margin, *(float(np.min(np.abs(c - t)) / c[-1]) for t in at))
    tok = [int(S[min(int(np.searchsorted(c, t, side="right")), len(S) - 1)]) for t in at]
    return tok, S, (x[S] - np.log(c[-1])).astype(np.float64), margin


def rows_agree(z, u, T=None, p=None):
    """z [N, V] float32 on the host."""
    N = z.shape[0]
    kn = {}
    if T is not None:
        kn["temperature"] = T
    if p is not None:
        kn["top_p"] = p
    o = run(torch.from_numpy(z).cuda(), u, **kn)
    off, ids, slq, tok = (t.cpu().numpy() for t in (o.offsets, o.ids, o.support_logq, o.tokens))
    for r in range(N):
        want, S, lq, margin = extended(z[r], [f32(v) for v in u[r]], f32(T[r]) if T is not None else 1.0, f32(p[r]) if p is not None else 1.0)
        assert margin > 2.0 ** -35, (r, math.log2(margin))
        if p is not None and p[r] < 1:
            assert off[r + 1] - off[r] == len(S), (r, off[r + 1] - off[r], len(S))
            np.testing.assert_array_equal(ids[off[r]:off[r + 1]], S, err_msg=f"row {r}")
            assert np.all(np.abs(slq[off[r]:off[r + 1]] - lq) <= 2.0 ** -23 * np.abs(lq) + 1e-9)
        np.testing.assert_array_equal(tok[r], want, err_msg=f"row {r}")
    assert o.status_bits() == 0, rh.status_names(o.status_bits())


@pytest.mark.parametrize("V", [(1 << 20) - 1, 1 << 20])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_constant_row_of_the_largest_vocabulary(V, dt):
    """2^20 weights of 1: the largest total there is.  The random numbers lie in the middle of a token's
    share (in 24 bits, so that they are the same in fp32)."""
    z = torch.zeros(2, V, dtype=dt, device="cuda")
    z[1] = -1.5
    u = (np.array([[0, 262144, 524288, (1 << 20) - 2], [1, 128974, 786432, 1047527]]) + 0.5) / (1 << 20)
    for kn in ({}, {"top_p": [0.5, 0.97]}, {"top_k": [700001, V - 1]}, {"min_p": [0.5, 1.0], "top_p": [0.25, 1.0]}):
        check(z, u, **kn)


def test_a_large_temperature_makes_a_flat_row():
    V = 1 << 20
    z = torch.randn(2, V, generator=torch.Generator().manual_seed(3)).cuda()
    check(z, np.array([[0.3, 0.9], [0.0, 0.6]]), temperature=[1e25, 1e25])


# tail logit, top_p: chosen so that the border keeps 2^-33 of the total away from the next
TIES = [(-21.0, 0.99995, 7), (-21.0, 0.9999, 7), (-22.2, 0.99998, 151935), (-22.2, 0.99997, 151935),
        (-12.5, 0.9, 0), (-12.5, 0.7, 0), (-18.0, 0.9995, 140000), (-18.0, 0.999, 140000)]


@pytest.mark.parametrize("tail,p,at", TIES)
def test_the_border_among_equal_logits_under_a_spike(tail, p, at):
    V = 151936
    z = np.full((1, V), tail, np.float32)
    z[0, at] = 0.0
    rows_agree(z, np.array([[0.25]]), p=[p])


# random numbers as multiples of 2^-24 from the top, and of 2^-30 and 2^-26 from 0
DRAWS = [
    (-14.0, [1 - 37 * 2.0 ** -24, 16 * 2.0 ** -30, 1 - 74 * 2.0 ** -24, 32 * 2.0 ** -30,
             1 - 111 * 2.0 ** -24, 48 * 2.0 ** -30, 1 - 148 * 2.0 ** -24, 64 * 2.0 ** -30]),
    (-18.0, [1 - 37 * 2.0 ** -24, 16 * 2.0 ** -30, 1 - 74 * 2.0 ** -24, 32 * 2.0 ** -30,
             1 - 111 * 2.0 ** -24, 48 * 2.0 ** -30, 1 - 148 * 2.0 ** -24, 64 * 2.0 ** -30]),
    (-20.0, [1 - 37 * 2.0 ** -24, 1 * 2.0 ** -30, 1 - 74 * 2.0 ** -24, 1 - 111 * 2.0 ** -24,
             3 * 2.0 ** -30, 1 - 148 * 2.0 ** -24, 4 * 2.0 ** -30, 1 - 185 * 2.0 ** -24]),
    (-21.5, [1 - 37 * 2.0 ** -24, 1 * 2.0 ** -30, 1 - 74 * 2.0 ** -24, 2 * 2.0 ** -30,
             1 - 111 * 2.0 ** -24, 1 - 148 * 2.0 ** -24, 4 * 2.0 ** -30, 5 * 2.0 ** -30]),
]


@pytest.mark.parametrize("tail,us", DRAWS)
def test_draws_from_a_flat_tail_under_spikes(tail, us):
    """Two likely tokens hold nearly all of the weight; the random numbers fall into the tail."""
    V = 151936
    z = np.full((1, V), tail, np.float32)
    z[0, 70001], z[0, 333] = 0.0, -2.0
    rows_agree(z, np.array([us]))


@pytest.mark.parametrize("seed,p", [(1, 0.999912934), (2, 0.99994391), (3, 0.999893606), (4, 0.999944823)])
def test_a_border_among_many_near_equal_logits(seed, p):
    """A tail of distinct logits in one bin of any coarse histogram."""
    V = 60000
    r = np.random.RandomState(seed)
    z = (-19 - 1e-3 * r.rand(1, V)).astype(np.float32)
    z[0, 5] = 0.0
    z[0, r.randint(0, V, 20)] = -3
    rows_agree(z, np.array([[0.5]]), p=[p])


@pytest.mark.parametrize("n", [3, 700, 5000, 20000])
def test_a_border_at_the_edge_of_a_stretch_of_logits(n):
    """n logits well above 40,000 others; top_p a little below, at and above the share of the n."""
    V = 60000
    r = np.random.RandomState(n)
    z = (-4 - 6 * r.rand(9, V)).astype(np.float32)
    at = r.permutation(V)[:n]
    z[:, at] = (0.5 * r.rand(9, n)).astype(np.float32)
    w = np.exp(z[0].astype(np.float64))
    z[:] = z[0]
    share = np.float32(w[at].sum() / w.sum())
    p = share + np.arange(-4, 5) * np.spacing(share)
    assert {len(extended(z[0], [0.5], 1.0, float(x))[1]) for x in p} == {n, n + 1}
    rows_agree(z, np.full((9, 1), 0.5), p=p)
