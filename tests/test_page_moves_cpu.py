"""Release, fork, compaction and copies of pages, host side: what is refused before any device work."""
import ctypes

import pytest
import torch

import lm_head_gb300 as rh
from lm_head_gb300 import pages as pg
from test_generation_cpu import FAKE, _fill, _refused, lib  # noqa: F401

ARG, UNS = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED
BIG = 1 << 31
WS = (FAKE, 1 << 40)


def test_struct_sizes():
    assert ctypes.sizeof(pg.RlPageReleaseArgs) == 15 * 8
    assert ctypes.sizeof(pg.RlPageForkArgs) == 17 * 8
    assert ctypes.sizeof(pg.RlPageCompactArgs) == 16 * 8
    assert ctypes.sizeof(pg.RlPageCopyArgs) == 8 * 8 + 5 * 4 + 4


def test_release_refusals(lib):  # noqa: F811
    def make(**kw):
        return _fill(pg.RlPageReleaseArgs, **{**dict(R=4, G=2, table_width=2, held_width=2, n_free=8, n_pages=8, page_size=16,
                                                     free_used_out=FAKE + 64), **kw})
    sizes = ("R", "G", "n_free", "n_pages", "table_width", "held_width")
    _refused(lib, "rl_page_release", make, [({s: -1}, ARG) for s in sizes] + [({s: BIG}, UNS) for s in sizes] + [
        (dict(page_size=0), UNS), (dict(page_size=8), UNS), (dict(kv_lens=None), ARG), (dict(keep_lens=None), ARG),
        (dict(block_table=None), ARG), (dict(held_lens=None), ARG), (dict(held_table=None), ARG), (dict(free_pages=None), ARG),
        (dict(free_used=None), ARG), (dict(free_used_out=None), ARG), (dict(free_used_out=FAKE), ARG)], tail=WS)
    a = make(n_pages=1 << 20)
    assert lib.rl_page_release(ctypes.byref(a), FAKE, 1 << 17, FAKE, None) == rh.RL_ERR_WORKSPACE
    assert lib.rl_page_release(ctypes.byref(a), None, 1 << 30, FAKE, None) == ARG
    assert lib.rl_page_release(ctypes.byref(a), FAKE + 8, 1 << 30, FAKE, None) == ARG
    assert lib.rl_page_release_workspace_bytes(1 << 20) >= 1 << 18 and lib.rl_page_release_workspace_bytes(-1) == 0


def test_fork_refusals(lib):  # noqa: F811
    at = dict(kv_lens=FAKE + (1 << 12), lens=FAKE + (2 << 12), parents=FAKE + (3 << 12), children=FAKE + (4 << 12),
              tokens=FAKE + (5 << 12))

    def make(**kw):
        return _fill(pg.RlPageForkArgs, **{**at, **dict(R=4, C=2, table_width=2, n_free=8, n_pages=8, page_size=16,
                                                        free_used_out=FAKE + 64), **kw})
    sizes = ("R", "C", "n_free", "n_pages", "table_width")
    _refused(lib, "rl_page_fork", make, [({s: -1}, ARG) for s in sizes] + [({s: BIG}, UNS) for s in sizes] + [
        (dict(page_size=48), UNS), (dict(parents=None), ARG), (dict(children=None), ARG), (dict(lens=None), ARG),
        (dict(kv_lens=None), ARG), (dict(block_table=None), ARG), (dict(free_pages=None), ARG), (dict(src=None), ARG),
        (dict(dst=None), ARG), (dict(tokens=None), ARG), (dict(free_used=None), ARG), (dict(free_used_out=FAKE), ARG),
        (dict(lens=at["kv_lens"] + 4), ARG), (dict(tokens=at["lens"]), ARG)], tail=WS)
    a = make(R=1000)
    assert lib.rl_page_fork(ctypes.byref(a), FAKE, 4000, FAKE, None) == rh.RL_ERR_WORKSPACE
    assert lib.rl_page_fork(ctypes.byref(a), None, 1 << 30, FAKE, None) == ARG


def test_fork_lists_that_share_memory(lib):  # noqa: F811
    apart = {n: FAKE + (k << 12) for k, n in enumerate(("kv_lens", "lens", "parents", "children", "src", "dst", "tokens"), 1)}

    def call(**kw):
        a = _fill(pg.RlPageForkArgs, **{**apart, **dict(R=4, C=2, table_width=2, n_free=8, n_pages=8, page_size=16,
                                                        free_used_out=FAKE + 64), **kw})
        return lib.rl_page_fork(ctypes.byref(a), *WS, FAKE, None)
    if not torch.cuda.is_available():
        assert call() not in (rh.RL_OK, ARG)                 # (no device)
    for x in ("parents", "children", "lens"):
        for y in ("kv_lens", "src", "dst", "tokens"):
            assert call(**{y: apart[x] + 4}) == ARG, (x, y)


def test_compact_refusals(lib):  # noqa: F811
    def make(**kw):
        return _fill(pg.RlPageCompactArgs, **{**dict(R=4, G=2, table_width=2, prefix_width=2, n_pages=8, page_size=16), **kw})
    sizes = ("R", "G", "n_pages", "table_width", "prefix_width")
    names = ("kv_lens", "block_table", "block_table_out", "prefix_lens", "prefix_table", "prefix_table_out", "src", "dst",
             "free_pages", "free_used_out")
    _refused(lib, "rl_page_compact", make, [({s: -1}, ARG) for s in sizes] + [({s: BIG}, UNS) for s in sizes] +
             [({n: None}, ARG) for n in names] + [(dict(page_size=17), UNS), (dict(block_table_out=FAKE + 4), ARG), (dict(prefix_table_out=FAKE + 4), ARG)],
             tail=WS)
    a = make(n_pages=1 << 20)
    assert lib.rl_page_compact(ctypes.byref(a), FAKE, 1 << 17, FAKE, None) == rh.RL_ERR_WORKSPACE
    assert lib.rl_page_compact(ctypes.byref(a), None, 1 << 30, FAKE, None) == ARG


def test_copy_refusals(lib):  # noqa: F811
    def make(**kw):
        return _fill(pg.RlPageCopyArgs, **{**dict(n=4, layer_stride=8 * 2 * 16 * 64, n_pages=8, layers=2, Hkv=2, D=64, page_size=16,
                                                  dtype=rh.RL_DTYPE_BF16), **kw})
    _refused(lib, "rl_page_copy", make, [
        (dict(n=-1), ARG), (dict(n_pages=-1), ARG), (dict(layers=-1), ARG), (dict(Hkv=0), ARG), (dict(D=0), ARG),
        (dict(page_size=9), UNS), (dict(dtype=7), UNS), (dict(n=BIG), UNS), (dict(layers=65537, layer_stride=1 << 40), UNS),
        (dict(layer_stride=8 * 2 * 16 * 64 - 1), ARG), (dict(layer_stride=-1), ARG), (dict(src=None), ARG), (dict(dst=None), ARG),
        (dict(k_cache=None), ARG), (dict(v_cache=FAKE + 8), ARG)])


def test_binding_refuses_host_tensors_and_shapes():
    i32 = torch.int32
    one, table = torch.ones(1, dtype=i32), torch.zeros(2, 3, dtype=i32)
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_release(torch.ones(2, dtype=i32), torch.ones(2, dtype=i32), table, one, one, page_size=16, n_pages=4)
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_fork(one, one, one, torch.ones(2, dtype=i32), table, one, one, page_size=16, n_pages=4)
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_compact(torch.ones(2, dtype=i32), table, page_size=16, n_pages=4)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_copy(one, one, cache, cache)
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_copy(one, one, cache, cache[:, :, :8])
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_copy(one, one, cache.to(torch.int16), cache.to(torch.int16))


class OnDevice:
    """A host tensor that says it lies on the device (for what the binding looks at before any device work)."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return OnDevice(self.t[i])


def test_copies_of_caches_with_layers_differently_far_apart(lib):  # noqa: F811
    """One call knows one distance between layers: a spaced cache beside a dense one is refused, whichever is which."""
    both = torch.zeros(3, 2, 5, 2, 16, 8, dtype=torch.bfloat16)
    spaced, dense, wider = both[:, 0], torch.zeros(3, 5, 2, 16, 8, dtype=torch.bfloat16), torch.zeros(3, 3, 5, 2, 16, 8, dtype=torch.bfloat16)[:, 1]
    none, status = OnDevice(torch.zeros(0, dtype=torch.int32)), OnDevice(torch.zeros(1, dtype=torch.int32))

    def call(k, v):
        with pytest.raises(rh.RLHeadError) as e:
            rh.rl_page_copy(none, none, OnDevice(k), OnDevice(v), status=status, stream=type("S", (), {"cuda_stream": 0}))
        return "dense layers" in str(e.value)
    assert call(spaced, dense) and call(dense, spaced) and call(spaced, wider)
    assert call(dense, dense.transpose(3, 4).contiguous().transpose(3, 4))
    if not torch.cuda.is_available():       # (what is sound gets as far as the missing device)
        assert not call(dense, dense) and not call(spaced, both[:, 1])
