"""Release, fork, compaction and copies of pages against plain loops (whole numbers and copies: every
value equal), with bad lengths, rows and ids among the inputs."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh

pytestmark = pytest.mark.gpu
ID_RANGE, LENGTHS, PAGES, PAGE_ID = 0x2, 0x400, 0x800, 0x1000


def dev(x, dtype=np.int32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def named(table, r, lo, hi, n_pages):
    """The page ids of a row's entries lo <= j < hi, and whether one was bad."""
    ids = [int(p) for p in table[r, lo:min(hi, table.shape[1])]]
    return {p for p in ids if 0 <= p < n_pages}, any(not 0 <= p < n_pages for p in ids)


def clip(n, W, page):
    """(entries, status bits) of a length."""
    if n < 0:
        return 0, LENGTHS
    e = -(-int(n) // page)
    return min(e, W), PAGES if e > W else 0


def release_reference(lens, keep, table, pool, used, page, n_pages, held_lens=None, held=None):
    bits, live, drop = 0, set(), set()
    R, W = table.shape
    for r in range(R):
        n, b = clip(lens[r], W, page)
        bits |= b
        k = int(keep[r])
        if k > max(int(lens[r]), 0):
            bits |= LENGTHS
            k = max(int(lens[r]), 0)
        m, b = clip(k, W, page)
        bits |= b
        for lo, hi, to in ((0, m, live), (m, n, drop)):
            ids, bad = named(table, r, lo, hi, n_pages)
            to |= ids
            bits |= PAGE_ID if bad else 0
    for g in range(0 if held is None else len(held_lens)):
        n, b = clip(held_lens[g], held.shape[1], page)
        ids, bad = named(held, g, 0, n, n_pages)
        live |= ids
        bits |= b | (PAGE_ID if bad else 0)
    back = sorted(drop - live)
    pool = pool.copy()
    if used < 0:
        bits |= LENGTHS
        used = 0
    base = used - len(back)
    bits |= PAGES if base < 0 or used > len(pool) else 0
    for i, p in enumerate(back):
        if 0 <= base + i < len(pool):
            pool[base + i] = p
    return pool, max(base, 0), bits


def check_release(lens, keep, table, pool, used, page, n_pages, held_lens=None, held=None):
    want, want_used, bits = release_reference(lens, keep, table, pool, used, page, n_pages, held_lens, held)
    d, t = dev(pool), dev(table)
    args = (dev(lens), dev(keep), t, d, dev([used]))
    kw = dict(page_size=page, n_pages=n_pages, held_lens=dev(held_lens), held_table=dev(held))
    o = rh.rl_page_release(*args, **kw)
    for _ in range(2):      # the same again gives the same
        np.testing.assert_array_equal(d.cpu().numpy(), want)
        assert int(o.free_used.item()) == want_used
        assert o.status_bits() == bits
        np.testing.assert_array_equal(t.cpu().numpy(), table)
        o.ws.fill_(255)
        o = rh.rl_page_release(*args, **kw, out=o)
    return bits


@pytest.mark.parametrize("R,len_max,page,shared,n_extra", [(1, 1, 16, 0, 0), (1, 5000, 16, 0, 3), (33, 300, 32, 0.5, 9),
                                                           (700, 513, 16, 0.3, 40), (4096, 900, 128, 0.9, 70000), (5, 90000, 16, 0.3, 1)])
def test_release(R, len_max, page, shared, n_extra):
    rng = np.random.default_rng(R * 7 + page)
    lens = rng.integers(0, len_max + 1, R)
    W = -(-len_max // page)
    n_pages = R * W + n_extra
    pool = rng.permutation(n_pages)
    table, used = np.full((R, W), -5), 0
    for r in range(R):
        n = -(-lens[r] // page)
        table[r, :n] = pool[used:used + n]
        used += n
        if r and rng.random() < shared:         # the first pages are the row's before
            s = rng.integers(0, min(lens[r], lens[r - 1]) // page + 1)
            table[r, :s] = table[r - 1, :s]
    keep = np.where(rng.random(R) < 0.3, lens, (lens * rng.random(R)).astype(int))
    assert check_release(lens, keep, table, pool, used, page, n_pages) == 0
    held = table[rng.integers(0, R, 3)].copy()
    held_lens = rng.integers(0, len_max + 1, 3)
    held[held < 0] = 0
    check_release(lens, keep, table, pool, used, page, n_pages, held_lens, held)


def test_release_bad_inputs():
    rng = np.random.default_rng(3)
    lens, page, n_pages = rng.integers(1, 200, 40), 16, 600
    table = rng.permutation(n_pages)[:40 * 13].reshape(40, 13)
    pool = rng.permutation(n_pages)
    keep = lens // 2
    assert check_release(lens, keep, table, pool, 520, page, n_pages) == 0
    for r, n, k in ((3, -7, 2), (4, 50, -1), (5, 50, 51), (6, 13 * 16 + 1, 13 * 16 + 1)):
        x, y = lens.copy(), keep.copy()
        x[r], y[r] = n, k
        assert check_release(x, y, table, pool, 520, page, n_pages) in (LENGTHS, PAGES)
    bad = table.copy()
    bad[::3, 0], bad[1::3, 1] = n_pages, -1
    assert check_release(lens, keep, bad, pool, 520, page, n_pages) == PAGE_ID
    assert check_release(lens, keep, table, pool, 5, page, n_pages) == PAGES         # more than were handed out
    assert check_release(lens, keep, table, pool, -3, page, n_pages) == LENGTHS | PAGES
    assert check_release(lens, keep, table, pool[:30], 520, page, n_pages) == PAGES     # used past the pool
    # the same page twice in a row, in a kept and a dropped entry of other rows
    twin = table.copy()
    twin[0, 5], twin[1, 9], lens[0], keep[0], lens[1], keep[1] = twin[0, 4], twin[0, 4], 160, 40, 200, 30
    assert check_release(lens, keep, twin, pool, 520, page, n_pages) == 0
    keep[1] = 200
    assert check_release(lens, keep, twin, pool, 520, page, n_pages) == 0


def test_release_nothing():
    z = np.zeros(0)
    assert check_release(z, z, np.zeros((0, 4), int), np.arange(9), 4, 16, 9) == 0
    assert check_release([0, 5], [0, 5], np.zeros((2, 0), int), np.arange(9), 4, 16, 9) == PAGES
    assert check_release([5], [0], np.array([[2]]), np.arange(3), 1, 16, 3) == 0


def fork_reference(par, chi, lens, kv, table, pool, used, page, n_pages):
    table, kv0, kv = table.copy(), kv, kv.copy()
    before = table.copy()
    R, W = table.shape
    C, bits = len(par), 0
    src, dst, tok = [-1] * C, [-1] * C, [0] * C
    if used < 0:
        used, bits = 0, LENGTHS
    first = {}
    for c in range(C):
        if 0 <= chi[c] < R:
            first.setdefault(int(chi[c]), c)
    for c in range(C):
        x, y, n = int(chi[c]), int(par[c]), int(lens[c])
        if not (0 <= x < R and 0 <= y < R) or first[x] != c or y in first:
            bits |= ID_RANGE
            continue
        if n < 0 or n > kv0[y]:
            bits |= LENGTHS
            continue
        if -(-n // page) > W:
            bits |= PAGES
            continue
        full, part = n // page, n % page
        row = [-1] * W
        for j in range(full):
            p = int(before[y, j])
            if 0 <= p < n_pages:
                row[j] = p
            else:
                bits |= PAGE_ID
        if part:
            s, d = int(before[y, full]), -1
            if used < len(pool):
                d = int(pool[used])
            else:
                bits |= PAGES
            used += 1
            if not 0 <= s < n_pages:
                bits |= PAGE_ID
                s = -1
            if used - 1 < len(pool) and not 0 <= d < n_pages:
                bits |= PAGE_ID
                d = -1
            row[full] = d
            if s >= 0 and d >= 0:
                src[c], dst[c], tok[c] = s, d, part
        table[x] = row
        kv[x] = n
    return dict(table=table, kv=kv, src=src, dst=dst, tok=tok, raw=used, bits=bits)


def check_fork(par, chi, lens, kv, table, pool, used, page, n_pages):
    want = fork_reference(par, chi, lens, kv, table, pool, used, page, n_pages)
    t, k = dev(table), dev(kv)
    args = (dev(par), dev(chi), dev(lens), k, t, dev(pool), dev([used]))
    o = rh.rl_page_fork(*args, page_size=page, n_pages=n_pages)
    for again in range(2):
        for name, got in (("table", t), ("kv", k), ("src", o.src), ("dst", o.dst), ("tok", o.tokens)):
            np.testing.assert_array_equal(got.cpu().numpy(), want[name], err_msg=name)
        assert int(o.free_used.item()) == min(want["raw"], max(max(used, 0), len(pool)))
        assert o.status_bits() == want["bits"]
        o.ws.fill_(again)
        o = rh.rl_page_fork(*args, page_size=page, n_pages=n_pages, out=o)
    return want["bits"]


def fork_case(R, C, len_max, page, seed):
    rng = np.random.default_rng(seed)
    W = -(-len_max // page)
    n_pages = R * W + C
    rows = rng.permutation(R)
    chi, old = rows[:C], rows[C:]
    par = rng.choice(old, C)
    kv = rng.integers(0, len_max + 1, R)
    lens = np.where(rng.random(C) < 0.5, kv[par], (kv[par] * rng.random(C)).astype(int))
    pool = rng.permutation(n_pages)
    table = pool[C:].reshape(R, W)
    return par, chi, lens, kv, table, pool, 0, page, n_pages


@pytest.mark.parametrize("R,C,len_max,page", [(2, 1, 1, 16), (9, 8, 64, 16), (300, 200, 700, 32), (5000, 4000, 90, 128), (6, 3, 70000, 16),
                                              (2048, 1500, 16, 16)])
def test_fork(R, C, len_max, page):
    assert check_fork(*fork_case(R, C, len_max, page, R)) == 0


def test_fork_bad_inputs():
    par, chi, lens, kv, table, pool, used, page, n_pages = fork_case(60, 30, 200, 16, 5)
    run = lambda **kw: check_fork(**{**dict(par=par, chi=chi, lens=lens, kv=kv, table=table, pool=pool, used=used, page=page,  # noqa: E731
                                            n_pages=n_pages), **kw})

    def put(a, i, v):
        a = a.copy()
        a[i] = v
        return a
    assert run() == 0
    assert run(chi=put(chi, 7, chi[2])) == ID_RANGE                 # twice a child: the first entry has it
    assert run(par=put(par, 7, chi[9])) == ID_RANGE                 # a parent that is a child
    assert run(par=put(par, 7, chi[7])) == ID_RANGE                 # its own parent
    assert run(chi=put(chi, 3, -1)) == ID_RANGE
    assert run(par=put(par, 3, 60)) == ID_RANGE
    assert run(lens=put(lens, 3, -1)) == LENGTHS
    assert run(lens=put(lens, 3, kv[par[3]] + 1)) == LENGTHS
    assert run(pool=pool[:5]) & PAGES                               # the pool runs out
    assert run(used=len(pool) - 3) & PAGES
    assert run(used=-2) == LENGTHS
    assert run(pool=put(pool, slice(0, 30), n_pages)) == PAGE_ID
    bad = table.copy()
    bad[:, ::2] = -1
    assert run(table=bad) & PAGE_ID
    wide = np.full(60, 16 * table.shape[1] + 40)
    assert run(kv=wide, lens=put(lens, 3, 16 * table.shape[1] + 17)) & PAGES
    z = np.zeros(0, int)
    assert run(par=z, chi=z, lens=z) == 0


def compact_reference(lens, table, n_pages, page, plens=None, ptable=None):
    live, bits, out = set(), 0, []
    pairs = [(lens, table)] + ([(plens, ptable)] if ptable is not None else [])
    for ln, t in pairs:
        for r in range(t.shape[0]):
            n, b = clip(ln[r], t.shape[1], page)
            ids, bad = named(t, r, 0, n, n_pages)
            live |= ids
            bits |= b | (PAGE_ID if bad else 0)
    n_live = len(live)
    goes = sorted(p for p in live if p >= n_live)
    holes = [p for p in range(n_live) if p not in live]
    to = dict(zip(goes, holes))
    assert len(goes) == len(holes)
    for ln, t in pairs:
        o = np.full(t.shape, -1)
        for r in range(t.shape[0]):
            for j in range(clip(ln[r], t.shape[1], page)[0]):
                p = int(t[r, j])
                o[r, j] = to.get(p, p) if 0 <= p < n_pages else -1
        out.append(o)
    pad = [-1] * (n_pages // 2 - len(goes))
    return out, goes + pad, holes + pad, n_live, bits


def check_compact(lens, table, n_pages, page, plens=None, ptable=None, in_place=False):
    out, src, dst, n_live, bits = compact_reference(lens, table, n_pages, page, plens, ptable)
    t, pt = dev(table), dev(ptable)
    kw = dict(page_size=page, n_pages=n_pages, prefix_lens=dev(plens), prefix_table=pt)
    o = rh.rl_page_compact(dev(lens), t, **kw)
    for again in range(2):
        np.testing.assert_array_equal(o.block_table.cpu().numpy(), out[0])
        if ptable is not None:
            np.testing.assert_array_equal(o.prefix_table.cpu().numpy(), out[1])
        np.testing.assert_array_equal(o.src.cpu().numpy(), src)
        np.testing.assert_array_equal(o.dst.cpu().numpy(), dst)
        np.testing.assert_array_equal(o.free_pages.cpu().numpy(), np.arange(n_pages))
        assert int(o.free_used.item()) == n_live and o.status_bits() == bits
        o.ws.fill_(77)
        if again == 0:          # and in place
            o.block_table = t
            if ptable is not None:
                o.prefix_table = pt
            o = rh.rl_page_compact(dev(lens), t, **kw, out=o)
    return bits


@pytest.mark.parametrize("R,G,len_max,page,spread", [(1, 0, 16, 16, 1.0), (1, 0, 1, 16, 40.0), (30, 4, 300, 32, 2.0), (600, 50, 500, 16, 1.2),
                                                     (3000, 1, 600, 128, 9.0), (2, 2, 40000, 16, 3.0)])
def test_compact(R, G, len_max, page, spread):
    rng = np.random.default_rng(R + G)
    W = -(-len_max // page)
    n_pages = int((R + G) * W * spread) + 1
    table = rng.permutation(n_pages)[:(R + G) * W].reshape(R + G, W)
    lens = rng.integers(0, len_max + 1, R + G)
    for r in range(1, R + G, 3):            # shared first pages
        table[r, :W // 2] = table[r - 1, :W // 2]
    if G:
        assert check_compact(lens[:R], table[:R], n_pages, page, lens[R:], table[R:]) == 0
    else:
        assert check_compact(lens, table, n_pages, page) == 0


def test_compact_bad_inputs_and_edges():
    rng = np.random.default_rng(9)
    table = rng.permutation(64)[:40].reshape(8, 5)
    lens = rng.integers(1, 81, 8)
    x = lens.copy()
    x[2], x[5] = -4, 81
    assert check_compact(x, table, 64, 16) == LENGTHS | PAGES
    bad = table.copy()
    bad[::2, 0], bad[1::2, 0] = 64, -2
    assert check_compact(lens, bad, 64, 16) == PAGE_ID
    assert check_compact(np.zeros(8, int), table, 64, 16) == 0                  # nothing lives
    assert check_compact(np.zeros(0, int), np.zeros((0, 3), int), 7, 16) == 0
    full = rng.permutation(40).reshape(8, 5)
    assert check_compact(np.full(8, 80), full, 40, 16) == 0                     # everything does
    assert check_compact(np.full(1, 16), np.array([[0]]), 1, 16) == 0           # one page: no list at all


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layers,Hkv,D,page", [(None, 2, 64, 16), (1, 1, 8, 128), (3, 8, 128, 64), (2, 3, 5, 32), (2, 1, 1, 16)])
def test_copy(dtype, layers, Hkv, D, page):
    g = torch.Generator(device="cuda").manual_seed(page + D)
    n_pages, n = 37, 15
    shape = (n_pages, Hkv, page, D) if layers is None else (layers, n_pages, Hkv, page, D)
    caches = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2)]
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    src[3], dst[5] = -1, -7
    src[6], dst[7] = n_pages, 1 << 30
    for tokens in (None, torch.randint(0, page + 1, (n,), generator=g, device="cuda", dtype=torch.int32)):
        bits = PAGE_ID
        if tokens is not None:
            tokens[0], tokens[1], tokens[2] = -3, page + 9, page
            bits |= LENGTHS
        want = [c.clone() for c in caches]
        for c in want:
            v = c if layers is not None else c[None]
            for i in range(n):
                s, d = int(src[i]), int(dst[i])
                if 0 <= s < n_pages and 0 <= d < n_pages:
                    k = page if tokens is None else min(max(int(tokens[i]), 0), page)
                    v[:, d, :, :k] = v[:, s, :, :k]
        got = [c.clone() for c in caches]
        st = rh.rl_page_copy(src, dst, *got, tokens=tokens)
        assert int(st.item()) == bits
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_copy_layers_apart():
    """Layers of a larger buffer, whose gap stays as it is; also one not a multiple of 16 bytes."""
    for gap in (64, 3):
        n_pages, Hkv, page, D = 6, 2, 16, 64
        one = n_pages * Hkv * page * D
        bufs = [torch.arange(3 * (one + gap), device="cuda").to(torch.bfloat16) + i for i in range(2)]
        view = lambda b: b.as_strided((3, n_pages, Hkv, page, D), (one + gap, Hkv * page * D, page * D, D, 1))  # noqa: E731
        want = [b.clone() for b in bufs]
        for w in want:
            view(w)[:, 4] = view(w)[:, 1].clone()
        i = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
        assert int(rh.rl_page_copy(i(1), i(4), view(bufs[0]), view(bufs[1])).item()) == 0
        assert torch.equal(bufs[0], want[0]) and torch.equal(bufs[1], want[1])


def test_copy_past_32_bits():
    """Pages whose bytes lie past 2^32 of their cache."""
    n_pages, Hkv, page, D = 40000, 4, 128, 128
    k = torch.zeros(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[39998], v[39998] = 3, 4
    i = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    assert int(rh.rl_page_copy(i(39998), i(39999), k, v).item()) == 0
    assert bool((k[39999] == 3).all()) and bool((v[39999] == 4).all()) and not bool(k[:39998].any())


def test_a_life_of_pages():
    """Prompts planned and written, rows forked and extended, half of them released, the rest moved together: every
    token stays readable through the tables, on a stream of its own and captured in a graph."""
    torch.manual_seed(1)
    page, R, W, n_pages, Hkv, D, L = 16, 12, 8, 200, 2, 64, 2
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = (torch.full((L, n_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    pool = torch.randperm(n_pages, device="cuda").to(torch.int32)
    log = [[] for _ in range(R)]            # what each row's tokens are

    def step(q, ctx, used):
        T = int(q.sum())
        p = rh.rl_page_plan(q, ctx, table, pool, page_size=page, n_pages=n_pages, n_tokens=T, free_used=used)
        new = torch.randn(L, T, Hkv, D, device="cuda").to(torch.bfloat16)
        for layer in range(L):
            rh.rl_kv_append(new[layer], -new[layer], p.slot_map, kc[layer], vc[layer])
        cu = p.cu_q.tolist()
        for r in range(R):
            log[r] += [new[:, t] for t in range(cu[r], cu[r + 1])]
        assert p.status_bits() == 0
        return p

    def look(lens, table, kc, vc):
        lens, t = lens.tolist(), table.tolist()
        for r in range(R):
            assert lens[r] == len(log[r])
            for j, x in enumerate(log[r]):
                pg = t[r][j // page]
                assert torch.equal(kc[:, pg, :, j % page], x) and torch.equal(vc[:, pg, :, j % page], -x)

    first = i32([37, 16, 50, 1] + [0] * 8)
    p = step(first, torch.zeros_like(first), i32([0]))
    kv = p.kv_lens
    par, chi, at = i32([0, 0, 1, 2, 3, 2]), i32([4, 5, 6, 7, 8, 9]), i32([37, 20, 16, 50, 1, 0])
    f = rh.rl_page_fork(par, chi, at, kv, table, pool, p.free_used, page_size=page, n_pages=n_pages)
    rh.rl_page_copy(f.src, f.dst, kc, vc, tokens=f.tokens, status=f.status)
    for c, (a, b, n) in enumerate(zip(par.tolist(), chi.tolist(), at.tolist())):
        log[b] = list(log[a][:n])
    assert f.status_bits() == 0
    look(kv, table, kc, vc)
    q = i32([3, 20, 1, 15, 7, 0, 16, 2, 30, 5, 0, 40])
    p2 = step(q, kv, f.free_used)
    look(p2.kv_lens, table, kc, vc)
    # rows 0, 2 and 4 end, others step back; captured
    keep = p2.kv_lens.clone()
    keep[[0, 2, 4]] = 0
    keep[8] -= 20
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rel = rh.rl_page_release(p2.kv_lens, keep, table, pool, p2.free_used, page_size=page, n_pages=n_pages, stream=s)
    com = rh.rl_page_compact(keep, table, page_size=page, n_pages=n_pages, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rh.rl_page_release(p2.kv_lens, keep, table, pool, p2.free_used, page_size=page, n_pages=n_pages, out=rel)
        rh.rl_page_compact(keep, table, page_size=page, n_pages=n_pages, out=com)
        rh.rl_page_copy(com.src, com.dst, kc, vc, status=com.status)
    g.replay()
    torch.cuda.synchronize()
    for r, n in enumerate(keep.tolist()):
        log[r] = log[r][:n]
    assert rel.status_bits() == 0 and com.status_bits() == 0
    used = int(rel.free_used.item())
    live = int(com.free_used.item())
    assert used == live                     # what is handed out is what lives: shared pages once
    # the pool's rest and the pages that rows name are all the pages, each once
    ids = {int(table[r, j]) for r, n in enumerate(keep.tolist()) for j in range(-(-n // page))}
    assert sorted(pool[used:].tolist() + list(ids)) == list(range(n_pages))
    look(keep, com.block_table, kc, vc)
    assert int(com.block_table.max()) < live
    # the same tables, lengths and pool go on
    table, pool = com.block_table, com.free_pages
    p3 = step(i32([18] * R), keep, com.free_used)
    look(p3.kv_lens, table, kc, vc)
