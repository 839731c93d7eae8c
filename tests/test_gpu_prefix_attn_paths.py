"""rl_prefix_attn on the paths that a step's shape picks: prefix and own keys in one block, many
groups, whole prompts, and each key's value by itself.

Bars as in test_gpu_prefix_attn.py.  Where one column holds a single key's value, all others zero,
the result is that key's weight times the value: the weight's and the result's rounding are
relative (half a step each, eps together; 2^-13 more for the fp32 exponent and sums), so that a
lost, doubled or misplaced value row shows in its column.
"""
import numpy as np
import pytest
import torch

from test_gpu_prefix_attn import BF, HF, Case
from test_gpu_prefix_attn_edges import BOTH

pytestmark = pytest.mark.gpu


def in_one_block(c):
    """Whether the call has no parts to join: then its rows run over prefix and own keys at once."""
    return c.run().ws.numel() == 1


@pytest.mark.parametrize("D,page,dtype", [(64, 16, BF), (128, 64, HF), (128, 128, BF), (64, 32, HF)])
def test_prefix_and_own_keys_in_one_block(D, page, dtype):
    """Ragged requests, some without tokens, some without a group or with an empty prefix; prefixes that
    end at, before and after a tile of 128 keys in the middle of a block's keys."""
    for prefixes in ([300, 50, 129, 1], [128, 0, 127, 256], [5, 700, 0, 1030]):
        c = Case(Hq=16, Hkv=2, D=D, page=page, dtype=dtype, seed=sum(prefixes), **{**BOTH, "prefixes": prefixes})
        assert in_one_block(c)
        c.check()


@pytest.mark.parametrize("G", [33, 64, 70, 200])
def test_many_groups_of_single_tokens(G):
    """Blocks find their group past the first 32, with groups of no, one and several requests."""
    groups = [(i * 7) % 4 for i in range(G)]
    R = sum(groups)
    Case(groups, [(i * 37) % 150 for i in range(G)], [1] * R, [1 + (i * 11) % 40 for i in range(R)], 8, 2, 64, 16, BF, G).check()


def test_many_groups_with_more_rows():
    """The same on tiles of up to 128 rows, and in one block."""
    groups = [9 if i % 5 else 14 for i in range(40)]
    R = sum(groups)
    Case(groups, [(i * 37) % 300 for i in range(40)], [1] * R, [1 + (i * 11) % 40 for i in range(R)], 8, 2, 64, 16, HF, 40).check()
    groups = [i % 3 for i in range(80)]
    R = sum(groups)
    q = [24 + (i * 13) % 30 for i in range(R)]
    q[5] = 129
    c = Case(groups, [(i * 53) % 200 for i in range(80)], q, [n + (i * 17) % 60 for i, n in enumerate(q)], 16, 2, 64, 16, BF, 41)
    assert in_one_block(c)
    c.check()


def causal_reference(c, r):
    """Request r's rows in 64 bits on the GPU, in slices of its tokens: out, lse, largest |v|."""
    R, Hq = len(c.q_lens), c.q.shape[1]
    k, v = c.keys[r]
    for g in range(len(c.groups)):
        if c.first[g] <= r < c.first[g + 1]:
            k, v = (torch.cat([a, b]) for a, b in zip(c.keys[R + g], (k, v)))
    k, v = (x.cuda().double().repeat_interleave(Hq // x.shape[1], 1) for x in (k, v))
    t0, n, m = sum(c.q_lens[:r]), c.q_lens[r], k.shape[0]
    out, lse = [], []
    for a in range(0, n, 512):
        b = min(n, a + 512)
        s = torch.einsum("qhd,khd->hqk", c.q[t0 + a:t0 + b].double(), k) * c.scale
        s.masked_fill_(torch.arange(m, device="cuda")[None] > (m - n + torch.arange(a, b, device="cuda"))[:, None], float("-inf"))
        lse.append(torch.logsumexp(s, 2).T)
        out.append(torch.einsum("hqk,khd->qhd", torch.softmax(s, 2), v))
    return torch.cat(out), torch.cat(lse), v.abs().amax()


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,n,ctx,prefix", [
    (2, 1, 64, 16, BF, 4096, 0, None), (4, 2, 128, 64, HF, 5003, 130, None), (2, 2, 128, 128, BF, 2500, 7, 1000),
    (8, 4, 64, 32, HF, 3001, 0, 200), (16, 2, 128, 64, BF, 8192, 0, None)])
def test_whole_prompts(Hq, Hkv, D, page, dtype, n, ctx, prefix):
    """A prompt of thousands of tokens in one step, beside a request of one token."""
    groups, prefixes = ([], []) if prefix is None else ([2], [prefix])
    c = Case(groups, prefixes, [n, 1], [n + ctx, 300], Hq, Hkv, D, page, dtype, n)
    a = c.run()
    assert a.status_bits() == 0
    eps = torch.finfo(dtype).eps
    for r in range(2):
        out, lse, vmax = causal_reference(c, r)
        rows = slice(0, n) if r == 0 else slice(n, n + 1)
        bar = eps / 2 * (out.abs() + vmax) + 2.0 ** -16 * vmax
        assert bool(((a.out[rows].double() - out).abs() <= bar).all())
        assert float((a.lse[rows].double() - lse).abs().max()) <= 2.0 ** -16


VALUES = [("warp", dict(groups=[2, 1], prefixes=[517, 64], q_lens=[1] * 3, kv_lens=[130, 700, 64])),
          ("keys", dict(groups=[17], prefixes=[700], q_lens=[1] * 17, kv_lens=[60 + 31 * i for i in range(17)])),
          ("keys, own", dict(groups=[], prefixes=[], q_lens=[20, 11], kv_lens=[1500, 400])),
          ("rows", dict(groups=[64], prefixes=[900], q_lens=[1] * 64, kv_lens=[40 + 7 * i for i in range(64)])),
          ("rows, own", dict(groups=[], prefixes=[], q_lens=[140, 70], kv_lens=[1000, 300])),
          ("one block", BOTH)]


@pytest.mark.parametrize("kind", [k for k, _ in VALUES])
@pytest.mark.parametrize("D,page,dtype", [(64, 16, BF), (128, 64, HF)])
def test_each_value_row_reaches_its_column(kind, D, page, dtype):
    """Column d holds the value of one key alone: the first D/2 columns keys of the prefix, the others keys
    of the request's own that its first token sees, spread over all of them with the last one among them."""
    c = Case(Hq=16, Hkv=2, D=D, page=page, dtype=dtype, seed=9, **dict(VALUES)[kind])
    c.q *= 0.3                                           # weights far above the least normal fp16
    R = len(c.q_lens)
    half = D // 2
    c.vc.zero_()
    for i, (k, v) in enumerate(c.keys):
        n = k.shape[0]
        seen = n if i >= R else n - c.q_lens[i] + 1      # by the request's first token
        v = torch.zeros_like(v)
        if seen > 0 and (i >= R or c.q_lens[i] > 0):
            at = np.unique(np.linspace(0, seen - 1, half).round().astype(int))
            cols = (half if i < R else 0) + np.arange(len(at))
            v[at, :, cols] = 64.0
        table = c.table[i] if i < R else c.ptable[i - R]
        for j in range(-(-n // page)):
            m = min(page, n - j * page)
            c.vc[int(table[j]), :, :m] = v[j * page:j * page + m].transpose(0, 1).cuda()
        c.keys[i] = (k, v)
    a = c.run()
    assert a.status_bits() == 0
    out, lse, _ = c.reference()
    got = a.out.cpu().double()
    eps = torch.finfo(dtype).eps
    assert bool(((got - out).abs() <= (eps + 2.0 ** -13) * out.abs()).all()), \
        float(((got - out).abs() / out.abs().clamp(min=1e-30)).max())
    assert bool((a.lse.cpu().double() - lse).abs().max() <= 2.0 ** -16)
