"""Page plans and cache writes against plain loops over the requests (whole numbers and copies:
every value equal)."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh

pytestmark = pytest.mark.gpu
LENGTHS, PAGES, PAGE_ID = 0x400, 0x800, 0x1000


def plan_reference(q, ctx, table, pool, used, page, n_pages, T, go=None, pl=None):
    """The plan request by request, with its status bits."""
    R, W = table.shape
    table = table.copy()
    cu, kv, slots, pos, bits = [0], [], [], [], 0
    for r in range(R):
        if q[r] < 0 or ctx[r] < 0:
            bits |= LENGTHS
        n, c = max(int(q[r]), 0), max(int(ctx[r]), 0)
        pre = 0
        if go is not None:
            for g in range(len(go) - 1):
                if go[g] <= r < go[g + 1]:
                    pre = max(int(pl[g]), 0)
        had, need = min(-(-c // page), W), min(-(-(c + n) // page), W)
        for j in range(had, need):
            ok = used < len(pool)
            bits |= 0 if ok else PAGES
            e = int(pool[used]) if ok else -1
            if ok and not 0 <= e < n_pages:
                bits |= PAGE_ID
                e = -1
            table[r, j] = e
            used += 1
        for i in range(n):
            at = c + i
            pg = -1
            if at // page >= W:
                bits |= PAGES
            else:
                pg = int(table[r, at // page])
                if at // page < had and not 0 <= pg < n_pages and len(slots) < T:
                    bits |= PAGE_ID
                    pg = -1
            slots.append(pg * page + at % page if pg >= 0 else -1)
            pos.append(pre + at)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    if cu[-1] != T:
        bits |= LENGTHS
    slots, pos = (np.asarray((x + [-1] * T)[:T]) for x in (slots, pos))
    return dict(cu_q=cu, kv_lens=kv, slot_map=slots, positions=pos, table=table, used=used, bits=bits)


def run_plan(q, ctx, table, pool, used, page, n_pages, T, go=None, pl=None):
    c = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    t = c(table)
    p = rh.rl_page_plan(c(q), c(ctx), t, c(pool), page_size=page, n_pages=n_pages, n_tokens=T,
                        free_used=None if used is None else c([used]), group_offsets=c(go), prefix_lens=c(pl))
    torch.cuda.synchronize()
    return p, t.cpu().numpy()


def check_plan(q, ctx, table, pool, used, page, n_pages, T, go=None, pl=None, want_bits=None):
    ref = plan_reference(q, ctx, table, pool, used or 0, page, n_pages, T, go, pl)
    p, t = run_plan(q, ctx, table, pool, used, page, n_pages, T, go, pl)
    np.testing.assert_array_equal(p.cu_q.cpu().numpy(), ref["cu_q"])
    np.testing.assert_array_equal(p.kv_lens.cpu().numpy(), ref["kv_lens"])
    np.testing.assert_array_equal(t, ref["table"])
    np.testing.assert_array_equal(p.slot_map.cpu().numpy(), ref["slot_map"])
    np.testing.assert_array_equal(p.positions.cpu().numpy(), ref["positions"])
    assert int(p.free_used.item()) == min(ref["used"], max(used or 0, len(pool)))
    assert p.status_bits() == ref["bits"], (rh.status_names(p.status_bits()), rh.status_names(ref["bits"]))
    if want_bits is not None:
        assert ref["bits"] == want_bits
    return ref


def make(R, q_max, ctx_max, page, seed, G=0):
    r = np.random.RandomState(seed)
    q, ctx = r.randint(0, q_max + 1, R), r.randint(0, ctx_max + 1, R)
    W = max(1, -(-(q_max + ctx_max) // page))
    n_pages = R * W + 5
    pool = r.permutation(n_pages)
    had = -(-ctx // page)
    table = np.full((R, W), -1)
    used = 0
    for i in range(R):
        table[i, :had[i]] = pool[used:used + had[i]]
        used += had[i]
    go = pl = None
    if G:
        go = np.concatenate([[0], np.sort(r.randint(0, R + 1, G - 1)), [R]])
        pl = r.randint(0, 500, G)
    return q, ctx, table, pool, used, page, n_pages, int(q.sum()), go, pl


@pytest.mark.parametrize("R,q_max,ctx_max,page,G", [
    (1, 1, 0, 16, 0), (1, 1, 5, 16, 1), (3, 1, 40, 16, 2), (128, 1, 300, 64, 16), (37, 33, 70, 32, 5), (255, 0, 9, 16, 3),
    (2047, 3, 40, 16, 100), (2048, 1, 17, 16, 2048), (2049, 5, 3, 128, 1), (5000, 4, 20, 16, 40), (9, 5000, 100, 64, 4)])
def test_plan_matches_loops(R, q_max, ctx_max, page, G):
    check_plan(*make(R, q_max, ctx_max, page, 100 + R, G), want_bits=0)


def test_plan_one_long_request_among_empty_ones():
    R, page = 300, 16
    q = np.zeros(R, int)
    q[150] = 20001
    W = -(-20001 // page)
    table = np.full((R, W), -1)
    check_plan(q, np.zeros(R, int), table, np.arange(W + 2)[::-1], None, page, W + 2, 20001, want_bits=0)


def test_plan_step_by_step_equals_one_plan():
    """Ten decode steps hand out the pages that one plan of ten tokens hands out when each
    request's pages are asked for in the same order (one request)."""
    page, W = 16, 4
    pool = np.random.RandomState(3).permutation(9)
    one = plan_reference([50], [0], np.full((1, W), -1), pool, 0, page, 9, 50)
    table, used, slots, ctx = np.full((1, W), -1), 0, [], 0
    for _ in range(50):
        p, table = run_plan([1], [ctx], table, pool, used, page, 9, 1)
        slots.append(int(p.slot_map.item()))
        used, ctx = int(p.free_used.item()), int(p.kv_lens.item())
    np.testing.assert_array_equal(slots, one["slot_map"])
    np.testing.assert_array_equal(table, one["table"])


def test_plan_bad_inputs_set_status_and_stay_in_bounds():
    page, W = 16, 3
    t = np.full((4, W), -1)
    # the pool runs out
    check_plan([20, 20, 20, 20], [0, 0, 0, 0], t, np.arange(5), None, page, 5, 80, want_bits=PAGES)
    # a row too short for its request
    check_plan([60, 1, 0, 2], [0, 0, 0, 0], t, np.arange(9), None, page, 9, 63, want_bits=PAGES)
    # negative lengths, and a sum that is not T (short and long)
    check_plan([3, -2, 4, 1], [0, 0, -7, 0], t, np.arange(9), None, page, 9, 8, want_bits=LENGTHS)
    check_plan([3, 2, 4, 1], [0, 0, 0, 0], t, np.arange(9), None, page, 9, 14, want_bits=LENGTHS)
    check_plan([3, 2, 4, 1], [0, 0, 0, 0], t, np.arange(9), None, page, 9, 6, want_bits=LENGTHS)
    # page ids outside the cache, in the pool and in the table
    check_plan([3, 2, 4, 1], [0, 0, 0, 0], t, [0, 99, -4, 2], None, page, 9, 10, want_bits=PAGE_ID)
    t2 = t.copy()
    t2[:, 0] = [4, 12, -1, 6]
    check_plan([3, 2, 4, 1], [1, 1, 1, 1], t2, np.arange(4), None, page, 9, 10, want_bits=PAGE_ID)


def test_plan_lengths_far_past_the_step():
    """Lengths whose sum passes T by far, up to 2^31 - 1 each: the call ends at once, the table holds
    what the rows have room for, and nothing past the buffers is written."""
    page, W, big = 16, 3, 2 ** 31 - 1
    t = np.full((5, W), -1)
    p, table = run_plan([big, 5, big, 7, big], [0, 0, big, 3, 17], t, np.arange(30), None, page, 30, 40)
    assert p.status_bits() & LENGTHS and p.status_bits() & PAGES
    np.testing.assert_array_equal(table[0], [0, 1, 2])
    np.testing.assert_array_equal(table[1], [3, -1, -1])
    assert p.slot_map.cpu().tolist() == list(range(40))


def test_plan_without_requests():
    p, _ = run_plan(np.zeros(0), np.zeros(0), np.zeros((0, 2)), np.arange(3), 2, 16, 3, 0)
    assert p.cu_q.tolist() == [0] and int(p.free_used.item()) == 2 and p.status_bits() == 0


# ---- cache writes --------------------------------------------------------------------

def append_reference(k, v, slot, kc, vc):
    page = kc.shape[2]
    kc, vc = kc.clone(), vc.clone()
    for t, s in enumerate(slot.tolist()):
        if 0 <= s < kc.shape[0] * page:
            kc[s // page, :, s % page] = k[t]
            vc[s // page, :, s % page] = v[t]
    return kc, vc


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,Hkv,D,page,layout", [
    (1, 1, 64, 16, "dense"), (5, 2, 128, 16, "dense"), (257, 4, 128, 64, "fused"), (300, 3, 64, 32, "fused"),
    (33, 2, 128, 128, "heads_first"), (17, 2, 72, 16, "odd"), (11, 1, 5, 16, "dense"), (40, 8, 128, 16, "broadcast")])
def test_append_matches_loops(T, Hkv, D, page, layout, dtype):
    g = torch.Generator().manual_seed(T)
    n_pages = T // page + 3
    if layout == "fused":
        x = torch.randn(T, 3 * Hkv, D, generator=g).to(dtype).cuda()
        k, v = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
    elif layout == "heads_first":
        k, v = (torch.randn(Hkv, T, D, generator=g).to(dtype).cuda().transpose(0, 1) for _ in range(2))
    elif layout == "odd":           # rows that no 16-byte load can start at
        x = torch.randn(T, Hkv, 2 * D + 3, generator=g).to(dtype).cuda()
        k, v = x[:, :, 1:D + 1], x[:, :, D + 2:2 * D + 2]
    elif layout == "broadcast":     # one token's values for all
        k, v = (torch.randn(1, Hkv, D, generator=g).to(dtype).cuda().expand(T, Hkv, D) for _ in range(2))
    else:
        k, v = (torch.randn(T, Hkv, D, generator=g).to(dtype).cuda() for _ in range(2))
    kc, vc = (torch.randn(n_pages, Hkv, page, D, generator=g).to(dtype).cuda() for _ in range(2))
    slot = torch.randperm(n_pages * page, generator=g)[:T]
    slot[torch.rand(T, generator=g) < 0.2] = -1
    slot = slot.cuda()
    rk, rv = append_reference(k, v, slot, kc, vc)
    st = rh.rl_kv_append(k, v, slot, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, rk) and torch.equal(vc, rv) and int(st.item()) == 0


def test_append_slots_outside_the_cache_are_left_out():
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()
    kc, vc = (torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slot = torch.tensor([3, 32, 1 << 40, -5], device="cuda")
    rk, rv = append_reference(k, k, slot, kc, vc)
    st = rh.rl_kv_append(k, k, slot, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, rk) and torch.equal(vc, rv) and int(st.item()) == PAGE_ID


def test_append_on_another_stream_and_empty():
    s = torch.cuda.Stream()
    k = torch.randn(4, 2, 64, device="cuda").half()
    kc, vc = (torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.float16) for _ in range(2))
    slot = torch.arange(4, device="cuda")
    torch.cuda.synchronize()
    st = rh.rl_kv_append(k, k, slot, kc, vc, stream=s)
    s.synchronize()
    assert torch.equal(kc[0, :, :4], k.transpose(0, 1)) and int(st.item()) == 0
    rh.rl_kv_append(k[:0], k[:0], slot[:0], kc, vc)
