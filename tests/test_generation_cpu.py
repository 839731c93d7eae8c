"""Generation operators, host side: arguments that are refused before any device work (no
GPU needed), and the binding's own checks."""
import ctypes

import pytest
import torch

import lm_head_gb300 as rh
from lm_head_gb300 import generation as gen

FAKE = 1 << 20          # 16-byte aligned, never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def lib():
    from lm_head_gb300 import build
    build.build()
    return rh.load()


def _fill(cls, **kw):
    a = cls()
    for name, typ in cls._fields_:
        if name in kw:
            setattr(a, name, kw[name])
        elif typ is ctypes.c_void_p:
            setattr(a, name, FAKE)
    return a


def _refused(lib, fn, make, changes, status=FAKE, tail=()):
    for change, want in changes:
        a = make(**change)
        assert getattr(lib, fn)(ctypes.byref(a), *tail, status, None) == want, change
    assert getattr(lib, fn)(None, *tail, status, None) == rh.RL_ERR_ARG
    good = make()
    assert getattr(lib, fn)(ctypes.byref(good), *tail, None, None) == rh.RL_ERR_ARG      # no status word


def test_struct_sizes():
    assert ctypes.sizeof(gen.RlPagePlanArgs) == 19 * 8
    assert ctypes.sizeof(gen.RlKvAppendArgs) == 11 * 8 + 4 * 4


def test_page_plan_refusals(lib):
    def make(**kw):
        return _fill(gen.RlPagePlanArgs, **{**dict(R=4, T=8, table_width=2, n_free=8, G=2, n_pages=8, page_size=16,
                                                   free_used_out=FAKE + 64), **kw})
    arg, uns = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED
    _refused(lib, "rl_page_plan", make, [
        (dict(R=-1), arg), (dict(T=-1), arg), (dict(G=-1), arg), (dict(n_free=-1), arg), (dict(n_pages=-1), arg),
        (dict(table_width=-1), arg), (dict(page_size=0), uns), (dict(page_size=24), uns), (dict(page_size=256), uns),
        (dict(R=1 << 31), uns), (dict(T=1 << 31), uns), (dict(n_pages=1 << 31), uns),
        (dict(q_lens=None), arg), (dict(ctx_lens=None), arg), (dict(block_table=None), arg), (dict(cu_q=None), arg),
        (dict(kv_lens=None), arg), (dict(slot_map=None), arg), (dict(free_pages=None), arg),
        (dict(group_offsets=None), arg), (dict(prefix_lens=None), arg), (dict(free_used_out=None), arg),
        (dict(free_used_out=FAKE), arg)])


def test_kv_append_refusals(lib):
    def make(**kw):
        return _fill(gen.RlKvAppendArgs, **{**dict(T=8, n_pages=4, Hkv=2, D=64, page_size=16, dtype=rh.RL_DTYPE_BF16), **kw})
    arg, uns = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED
    _refused(lib, "rl_kv_append", make, [
        (dict(T=-1), arg), (dict(n_pages=-1), arg), (dict(Hkv=0), arg), (dict(D=0), arg), (dict(page_size=17), uns),
        (dict(dtype=rh.RL_DTYPE_F32), uns), (dict(dtype=9), uns), (dict(T=1 << 31), uns), (dict(k=None), arg),
        (dict(v=None), arg), (dict(slot_map=None), arg), (dict(k_cache=None), arg), (dict(v_cache=FAKE + 8), arg)])


def test_binding_refuses_host_tensors_and_wrong_types():
    i32 = torch.int32
    with pytest.raises(rh.RLHeadError):
        rh.rl_page_plan(torch.ones(2, dtype=i32), torch.ones(2, dtype=i32), torch.zeros(2, 3, dtype=i32),
                        torch.arange(9, dtype=i32), page_size=16, n_pages=9, n_tokens=2)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(rh.RLHeadError):
        rh.rl_kv_append(k, k, torch.zeros(3, dtype=torch.int64), cache, cache)
    with pytest.raises(rh.RLHeadError):
        rh.rl_kv_append(k, k, torch.zeros(3, dtype=torch.int64), cache, cache[:, :, :8])


def test_sample_refusals(lib):
    def make(**kw):
        return _fill(gen.RlSampleArgs, **{**dict(N=4, V=1000, row_stride=1000, dtype=rh.RL_DTYPE_F32, K=2, capacity=10), **kw})
    arg, uns = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED
    _refused(lib, "rl_sample", make, [
        (dict(N=-1), arg), (dict(V=0), arg), (dict(K=0), arg), (dict(capacity=-1), arg), (dict(K=1025), uns),
        (dict(V=(1 << 20) + 1, row_stride=1 << 21), uns), (dict(dtype=3), uns), (dict(row_stride=999), arg),
        (dict(logits=None), arg), (dict(u=None), arg), (dict(tokens=None), arg), (dict(ids=None), arg),
        (dict(support_logq=None), arg), (dict(logits=FAKE + 2), arg)], tail=(FAKE, 1 << 30))
    a = make()
    assert lib.rl_sample(ctypes.byref(a), FAKE, 64, FAKE, None) == rh.RL_ERR_WORKSPACE
    assert lib.rl_sample(ctypes.byref(a), None, 1 << 30, FAKE, None) == rh.RL_ERR_ARG
    assert rh.rl_sample_workspace_bytes(4, 1000, 2) > 0 and rh.rl_sample_workspace_bytes(4, 1 << 21, 2) == 0
    assert ctypes.sizeof(gen.RlSampleArgs) == 17 * 8


def test_prefix_attn_refusals(lib):
    def make(**kw):
        return _fill(gen.RlPrefixAttnArgs, **{**dict(q_stride_t=256, q_stride_h=64, n_pages=8, T=4, R=2, G=1, table_width=2,
                                                     prefix_width=2, max_q=2, max_kv=32, max_prefix=32, Hq=4, Hkv=2, D=64,
                                                     page_size=16, dtype=rh.RL_DTYPE_BF16, scale=0.1), **kw})
    arg, uns = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED
    _refused(lib, "rl_prefix_attn", make, [
        (dict(T=-1), arg), (dict(R=-1), arg), (dict(G=-1), arg), (dict(max_kv=-1), arg), (dict(max_prefix=-1), arg),
        (dict(Hq=3), arg), (dict(Hkv=0), arg), (dict(D=96), uns), (dict(page_size=48), uns), (dict(dtype=0), uns),
        (dict(T=1 << 30), uns), (dict(n_pages=1 << 27), uns), (dict(max_q=0), arg), (dict(scale=float("nan")), arg), (dict(scale=-0.1), arg), (dict(scale=-0.1), arg),
        (dict(q=None), arg), (dict(out=None), arg), (dict(cu_q=None), arg), (dict(kv_lens=None), arg),
        (dict(block_table=None), arg), (dict(group_offsets=None), arg), (dict(prefix_lens=None), arg),
        (dict(prefix_table=None), arg), (dict(k_cache=None), arg), (dict(v_cache=FAKE + 2), arg), (dict(q=FAKE + 2), arg),
        (dict(q_stride_t=255), arg), (dict(q_stride_h=60), arg), (dict(n_pages=0), arg)], tail=(FAKE, 1 << 40))
    a = make()
    assert lib.rl_prefix_attn(ctypes.byref(a), FAKE, 16, FAKE, None) == rh.RL_ERR_WORKSPACE
    assert lib.rl_prefix_attn(ctypes.byref(a), None, 1 << 40, FAKE, None) == rh.RL_ERR_ARG
    bad = make(D=96)
    assert lib.rl_prefix_attn_workspace_bytes(ctypes.byref(bad)) == 0
    assert ctypes.sizeof(gen.RlPrefixAttnArgs) == 22 * 8 + 6 * 4
