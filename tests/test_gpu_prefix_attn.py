"""rl_prefix_attn against softmax attention in 64 bits.

Bars, for |v| <= vmax over the row's keys: the weights are rounded to the cache's type (half a
step, eps/2 of each: at most eps/2 * vmax after normalisation), and so is the output (eps/2 of its
value); fp32 products, sums and exponentials add below 2^-16 of vmax at these lengths (D 2^-24 for
the scores times |s| <= 64, plus the hardware exponential's 2^-22).  lse: the scores' error,
2^-24 D max|q||k| scale at most here 2^-16 absolute.
"""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh

pytestmark = pytest.mark.gpu
LENGTHS, PAGE_ID = 0x400, 0x1000


class Case:
    """A step over a paged cache: group sizes, prefix lengths, per-request (q_len, kv_len)."""

    def __init__(self, groups, prefixes, q_lens, kv_lens, Hq, Hkv, D, page, dtype, seed, stray=0, junk=float("nan")):
        g = torch.Generator().manual_seed(seed)
        R, G = len(q_lens), len(groups)
        self.q_lens, self.kv, self.prefixes, self.groups = list(q_lens), list(kv_lens), list(prefixes), list(groups)
        self.first = [stray + sum(groups[:i]) for i in range(G + 1)]
        W = max(1, max((-(-x // page) for x in kv_lens), default=1))
        WP = max(1, max((-(-x // page) for x in prefixes), default=1))
        n_pages = R * W + G * WP + 2
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        table, ptable = perm[:R * W].view(R, W).clone(), perm[R * W:R * W + G * WP].view(G, WP).clone()
        kc, vc = (torch.full((n_pages, Hkv, page, D), junk).to(dtype) for _ in range(2))
        self.keys = []
        for t, lens in ((table, kv_lens), (ptable, prefixes)):
            for r, n in enumerate(lens):
                k, v = (torch.randn(n, Hkv, D, generator=g).to(dtype) for _ in range(2))
                for c, x in ((kc, k), (vc, v)):
                    for j in range(-(-n // page)):
                        m = min(page, n - j * page)
                        c[t[r, j].item(), :, :m] = x[j * page:j * page + m].transpose(0, 1)
                self.keys.append((k, v))
                t[r, -(-n // page):] = -1                     # what no length reaches is never looked at
        T = sum(q_lens)
        self.q = torch.randn(T, Hq, D, generator=g).to(dtype).cuda()
        self.kc, self.vc = kc.cuda(), vc.cuda()
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cu = i([0] + list(np.cumsum(q_lens)))
        self.kvt, self.table, self.ptable = i(list(kv_lens)), table.cuda(), ptable.cuda()
        self.go, self.pl = i(self.first), i(list(prefixes))
        self.scale = D ** -0.5
        self.bounds = dict(max_q=max(list(q_lens) + [1]), max_kv=max(list(kv_lens) + [0]), max_prefix=max(list(prefixes) + [0]))

    def run(self, q=None, **kw):
        b = {**self.bounds, **kw}
        grouped = {} if not self.groups else dict(group_offsets=self.go, prefix_lens=self.pl, prefix_table=self.ptable)
        if not self.groups:
            b.pop("max_prefix")
        a = rh.rl_prefix_attn(self.q if q is None else q, self.kc, self.vc, self.cu, self.kvt, self.table, scale=self.scale,
                              **grouped, **b)
        torch.cuda.synchronize()
        return a

    def reference(self):
        T, Hq, D = self.q.shape
        R = len(self.q_lens)
        out, lse, vmax = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -float("inf"), dtype=torch.float64), torch.zeros(T, Hq)
        cu = np.cumsum([0] + self.q_lens)
        q = self.q.cpu().double()
        for r in range(R):
            n, L = self.q_lens[r], self.kv[r]
            k, v = (x.double() for x in self.keys[r])
            P = 0
            for g in range(len(self.groups)):
                if self.first[g] <= r < self.first[g + 1]:
                    pk, pv = (x.double() for x in self.keys[R + g])
                    P = pk.shape[0]
                    k, v = torch.cat([pk, k]), torch.cat([pv, v])
            Hkv = k.shape[1]
            for i in range(n):
                m = P + L - n + i + 1
                if m == 0:
                    continue
                kk, vv = (x[:m].repeat_interleave(Hq // Hkv, 1) for x in (k, v))
                s = torch.einsum("hd,khd->hk", q[cu[r] + i], kk) * self.scale
                lse[cu[r] + i] = torch.logsumexp(s, 1)
                out[cu[r] + i] = torch.einsum("hk,khd->hd", torch.softmax(s, 1), vv)
                vmax[cu[r] + i] = vv.abs().amax((0, 2))
        return out, lse, vmax

    def check(self, a=None, **kw):
        a = self.run(**kw) if a is None else a
        out, lse, vmax = self.reference()
        eps = torch.finfo(self.q.dtype).eps
        got, gl = a.out.cpu().double(), a.lse.cpu().double()
        bar = eps / 2 * (out.abs() + vmax[..., None]) + 2.0 ** -16 * vmax[..., None]
        assert bool(((got - out).abs() <= bar).all()), float(((got - out).abs() / bar.clamp(min=1e-30)).max())
        assert torch.equal(torch.isinf(gl), torch.isinf(lse))
        f = torch.isfinite(lse)
        assert bool(((gl[f] - lse[f]).abs() <= 2.0 ** -16).all())
        assert a.status_bits() == 0, rh.status_names(a.status_bits())
        return a


BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("D,page,dtype", [(64, 16, BF), (128, 32, HF), (128, 64, BF), (64, 128, HF)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (6, 2), (20, 4), (40, 2)])
def test_one_token_steps(Hq, Hkv, D, page, dtype):
    Case([3, 1, 4], [70, 0, 333], [1] * 8, [1, 17, 64, 65, 129, 300, 2, 128], Hq, Hkv, D, page, dtype, 1).check()


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000, 4097])
def test_lengths(n):
    Case([1, 2], [n, max(n - 1, 0)], [1, 1, 1], [1, n, max(n - 2, 1)], 4, 2, 64, 16, BF, n).check()
    Case([], [], [1, 1], [n, 1], 4, 2, 128, 64, HF, n).check()


@pytest.mark.parametrize("q_lens", [[2, 3, 1, 0, 5], [0, 0, 1, 0, 0], [40, 1, 17, 0, 100], [130, 257, 3, 64, 16]])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (5, 1, 128, 64), (16, 2, 128, 32)])
def test_steps_of_several_tokens_are_causal(q_lens, Hq, Hkv, D, page):
    kv = [n + x for n, x in zip(q_lens, [0, 9, 0, 33, 200])]
    for dtype in (BF, HF):
        Case([2, 3], [37, 150], q_lens, kv, Hq, Hkv, D, page, dtype, sum(q_lens)).check()


@pytest.mark.parametrize("prefix", [1, 63, 127, 128, 129, 256, 257, 383, 1000, 2050])
@pytest.mark.parametrize("groups,Hq,Hkv,D,page", [([17], 1, 1, 64, 16), ([8, 8], 8, 2, 128, 32), ([33], 8, 2, 128, 64),
                                                  ([16, 40], 12, 2, 64, 128), ([64], 16, 2, 128, 16)])
def test_many_rows_share_a_prefix(groups, Hq, Hkv, D, page, prefix):
    """17 to 512 query rows of a key head over a prefix that ends at, before and after a tile; own
    lengths from one."""
    R = sum(groups)
    kv = [1 + (7 * i) % 70 for i in range(R)]
    Case(groups, [max(prefix - 5 * i, 1) for i in range(len(groups))], [1] * R, kv, Hq, Hkv, D, page,
         BF if D == 128 else HF, prefix + R).check()


@pytest.mark.parametrize("n", [9, 32, 33, 64, 65, 128, 129, 300])
def test_a_long_step_of_one_request(n):
    """Causal tiles: rows 18 to 600, with and without cached keys, without a prefix."""
    for ctx in (0, 1, 127, 200):
        Case([], [], [n], [n + ctx], 2, 1, 64, 64, BF, n + ctx).check()
    Case([1], [129], [n], [n + 77], 4, 2, 128, 16, HF, n).check()


def test_requests_outside_groups_and_groups_without_requests():
    Case([0, 2, 0, 1], [64, 50, 9, 100], [1, 2, 1, 1, 3], [5, 2, 40, 1, 3], 8, 4, 128, 16, BF, 3, stray=1).check()


def test_rows_that_see_nothing():
    c = Case([2, 1], [0, 20], [1, 1, 1], [1, 1, 1], 4, 2, 64, 16, BF, 4)
    c.kv = [0, 1, 0]
    c.kvt = torch.tensor(c.kv, dtype=torch.int32, device="cuda")
    c.keys[0], c.keys[2] = ((x[:0] for x in c.keys[i]) for i in (0, 2))
    c.keys = [tuple(k) for k in c.keys]
    a = c.run()
    assert bool((a.out[0] == 0).all()) and bool(torch.isinf(a.lse[0]).all())
    assert bool(torch.isfinite(a.out).all()) and a.status_bits() == LENGTHS       # a step token without its own key


def test_padding_rows_are_zero():
    for groups, prefixes in (([2], [30]), ([], [])):
        c = Case(groups, prefixes, [1, 2], [4, 9], 4, 2, 64, 16, BF, 5)
        q = torch.cat([c.q, torch.full((5, 4, 64), float("nan"), device="cuda", dtype=BF)])
        a = c.run(q)
        assert bool((a.out[3:] == 0).all()) and bool((a.lse[3:] == -float("inf")).all())
        ref, _, _ = c.reference()
        assert bool(torch.isfinite(a.out[:3]).all()) and float((a.out[:3].cpu().double() - ref).abs().max()) < 0.05


def test_infinities_and_large_scores():
    """Scores of several hundred (fp32 exponents must not overflow), and junk of infinities past the
    lengths."""
    c = Case([2], [100], [1, 1], [33, 64], 4, 2, 128, 16, HF, 6, junk=float("inf"))
    c.q *= 16
    a = c.run()
    out, lse, vmax = c.reference()
    assert bool(torch.isfinite(a.out).all()) and float(lse.max()) > 30
    # scores 16 times as large: their fp32 error is, too
    bar = torch.finfo(HF).eps / 2 * (out.abs() + vmax[..., None]) + 2.0 ** -12 * vmax[..., None]
    assert bool(((a.out.cpu().double() - out).abs() <= bar).all())
    assert float((a.lse.cpu().double() - lse).abs().max()) <= 2.0 ** -12


def test_strided_queries():
    c = Case([2], [40], [3, 2], [10, 5], 8, 2, 64, 16, BF, 7)
    want = c.check()
    x = torch.zeros(5, 3, 8, 64, device="cuda", dtype=BF)
    x[:, 1] = c.q
    for q in (x[:, 1], c.q.transpose(0, 1).contiguous().transpose(0, 1)):
        a = c.run(q)
        assert torch.equal(a.out, want.out) and torch.equal(a.lse, want.lse)


def test_bounds_above_the_lengths_change_nothing_that_matters():
    """Larger bounds cut the keys into other parts: the same results to rounding."""
    c = Case([3], [500], [1, 1, 1], [90, 700, 3], 8, 2, 128, 64, BF, 8)
    c.check()
    c.check(max_kv=20000 // 64 * 64, max_q=4, max_prefix=30000)


def test_bad_lengths_and_pages_set_status():
    c = Case([2], [40], [1, 1], [20, 30], 4, 2, 64, 16, BF, 9)
    t = c.table.clone()
    c.table[1, 1] = 10 ** 6
    assert c.run().status_bits() == PAGE_ID
    c.table[1, 1] = -3
    assert c.run().status_bits() == PAGE_ID
    c.table = t
    assert c.run(max_kv=16).status_bits() == LENGTHS
    assert c.run(max_prefix=16).status_bits() == LENGTHS
    good = c.cu
    for cu in ([0, 1, 100], [0, -5, 2], [0, 2, 1], [1, 1, 2]):
        c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert c.run().status_bits() & LENGTHS
    c.cu = good
    c.pl = torch.tensor([-4], dtype=torch.int32, device="cuda")
    assert c.run().status_bits() == LENGTHS
    c.pl = torch.tensor([10 ** 9], dtype=torch.int32, device="cuda")
    assert c.run().status_bits() == LENGTHS


def test_a_short_wait_limit_is_an_error_not_a_fault():
    """A wait that runs out sets TIMEOUT and the kernel returns (limit: 1 us)."""
    c = Case([4], [5000], [1] * 4, [900] * 4, 8, 2, 128, 16, BF, 10)
    want = c.run()
    rh.rl_set_option(rh.RL_OPT_WAIT_LIMIT_US, 1)
    try:
        bits = c.run().status_bits()
    finally:
        rh.rl_set_option(rh.RL_OPT_WAIT_LIMIT_US, 1_000_000)
    assert bits & ~0x200 == 0
    again = c.run()
    assert again.status_bits() == 0 and torch.equal(again.out, want.out)


def test_repeats_are_bitwise_equal_and_a_graph_replays_with_new_lengths():
    c = Case([4, 4], [1000, 77], [1] * 8, [300, 5, 64, 200, 9, 512, 33, 1], 16, 4, 128, 64, BF, 11)
    a, b = c.run(), c.run()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    kw = dict(group_offsets=c.go, prefix_lens=c.pl, prefix_table=c.ptable, scale=c.scale, **c.bounds)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o = rh.rl_prefix_attn(c.q, c.kc, c.vc, c.cu, c.kvt, c.table, **kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rh.rl_prefix_attn(c.q, c.kc, c.vc, c.cu, c.kvt, c.table, out=o, **kw)
    c.kv = [x - (x > 1) for x in c.kv]
    c.kvt.copy_(torch.tensor(c.kv, dtype=torch.int32))
    c.keys = [tuple(x[:n] for x in k) for k, n in zip(c.keys, c.kv)] + c.keys[8:]
    g.replay()
    torch.cuda.synchronize()
    c.check(o)
