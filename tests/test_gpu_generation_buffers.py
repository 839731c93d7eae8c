"""The generation operators' own buffers: workspaces with any contents, and what a call on another
stream makes."""
import pytest
import torch

import lm_head_gb300 as rh

pytestmark = pytest.mark.gpu


def sampling_inputs(N=40, V=5000):
    g = torch.Generator().manual_seed(4)
    z = (3 * torch.randn(N, V, generator=g)).cuda()
    top_p = torch.full((N,), 0.9, device="cuda")
    top_p[::3] = 1.0
    return z, torch.rand(N, 5, generator=g).cuda(), top_p


@pytest.mark.parametrize("fill", [0, 1, 255])
def test_a_sampling_workspace_may_hold_anything(fill):
    z, u, top_p = sampling_inputs()
    want = rh.rl_sample(z, u, top_p=top_p, capacity=z.numel())
    n = rh.rl_sample_workspace_bytes(*z.shape, u.shape[1])
    for _ in range(2):          # a workspace that was just used, too
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            o = rh.rl_sample(z, u, top_p=top_p, capacity=z.numel(), ws=ws)
            assert torch.equal(o.offsets, want.offsets) and torch.equal(o.tokens, want.tokens)
            assert torch.equal(o.ids, want.ids) and torch.equal(o.support_logq, want.support_logq)
            assert o.status_bits() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_plan_and_append_on_another_stream_keep_their_status():
    q, ctx, table, pool = i32([3, -1]), i32([0, 0]), torch.full((2, 1), -1, dtype=torch.int32, device="cuda"), i32([0, 1])
    k = torch.ones(3, 2, 64, device="cuda").bfloat16()
    cache = [torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    slots = torch.tensor([0, 1, 999], device="cuda")
    s = torch.cuda.Stream()
    for _ in range(2):          # the first time kernels are loaded, which takes longer than the sleep
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        p = rh.rl_page_plan(q, ctx, table, pool, page_size=16, n_pages=2, n_tokens=3, stream=s)
        st = rh.rl_kv_append(k, k, slots, *cache, stream=s)
    torch.cuda.synchronize()
    assert p.status_bits() == 0x400 and int(st.item()) == 0x1000
    assert p.slot_map.tolist() == [0, 1, 2]


def test_attention_on_another_stream():
    from test_gpu_prefix_attn import BF, Case
    c = Case([3], [70], [1] * 3, [1, 17, 64], 8, 2, 64, 16, BF, 1)
    want = c.check()
    c.bounds["max_kv"] = 32
    s = torch.cuda.Stream()
    kw = dict(group_offsets=c.go, prefix_lens=c.pl, prefix_table=c.ptable, scale=c.scale, max_q=1, max_prefix=70)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    a = rh.rl_prefix_attn(c.q, c.kc, c.vc, c.cu, c.kvt, c.table, max_kv=32, stream=s, **kw)
    b = rh.rl_prefix_attn(c.q, c.kc, c.vc, c.cu, c.kvt, c.table, max_kv=64, stream=s, **kw)
    torch.cuda.synchronize()
    assert a.status_bits() == 0x400 and b.status_bits() == 0
    assert torch.equal(b.out, want.out) and torch.equal(b.lse, want.lse)


def test_sampling_on_another_stream():
    z, u, top_p = sampling_inputs()
    u[3, 2] = 1.5
    want = rh.rl_sample(z, u, top_p=top_p, capacity=z.numel())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    o = rh.rl_sample(z, u, top_p=top_p, capacity=z.numel(), stream=s)
    torch.cuda.synchronize()
    assert o.status_bits() == want.status_bits() == 0x2000
    n = want.nnz()
    assert n == o.nnz() and torch.equal(o.tokens, want.tokens) and torch.equal(o.ids[:n], want.ids[:n])
    assert torch.equal(o.support_logq[:n], want.support_logq[:n])
