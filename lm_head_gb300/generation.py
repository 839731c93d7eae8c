"""Binding of the generation operators (include/rlhead.h, "generation"): page plans, cache
writes, attention over a shared prefix, and sampling with the head's support rows.

Argument marshalling only, as in the package's other calls.  Every function takes its output
buffers through `out` / `status`, so that a decode loop allocates nothing after its first step
(and can be captured in a CUDA graph); without them it makes them.  The status word is
never cleared by the library: read it with status_bits() and zero it.  With stream=, what a call
makes is made on that stream, as under torch.cuda.stream(stream).
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import struct
import sys
from typing import Optional

import torch

RL_DTYPE_F32, RL_DTYPE_BF16, RL_DTYPE_F16 = 0, 1, 2
_DTYPES = {torch.float32: RL_DTYPE_F32, torch.bfloat16: RL_DTYPE_BF16, torch.float16: RL_DTYPE_F16}
_P, _I64, _I32, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class RlPagePlanArgs(ctypes.Structure):
    _fields_ = [("R", _I64), ("T", _I64), ("q_lens", _P), ("ctx_lens", _P), ("block_table", _P),
                ("table_width", _I64), ("free_pages", _P), ("n_free", _I64), ("free_used", _P),
                ("free_used_out", _P), ("group_offsets", _P), ("prefix_lens", _P), ("G", _I64), ("n_pages", _I64),
                ("page_size", _I32), ("cu_q", _P), ("kv_lens", _P), ("slot_map", _P), ("positions", _P)]


class RlKvAppendArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_stride_t", _I64), ("k_stride_h", _I64), ("v_stride_t", _I64),
                ("v_stride_h", _I64), ("slot_map", _P), ("k_cache", _P), ("v_cache", _P), ("T", _I64),
                ("n_pages", _I64), ("Hkv", _I32), ("D", _I32), ("page_size", _I32), ("dtype", _I32)]


class RlPrefixAttnArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("q_stride_t", _I64), ("q_stride_h", _I64), ("k_cache", _P), ("v_cache", _P),
                ("n_pages", _I64), ("T", _I64), ("R", _I64), ("G", _I64), ("cu_q", _P), ("kv_lens", _P),
                ("block_table", _P), ("table_width", _I64), ("group_offsets", _P), ("prefix_lens", _P),
                ("prefix_table", _P), ("prefix_width", _I64), ("max_q", _I64), ("max_kv", _I64), ("max_prefix", _I64),
                ("Hq", _I32), ("Hkv", _I32), ("D", _I32), ("page_size", _I32), ("dtype", _I32), ("scale", _F),
                ("out", _P), ("lse", _P)]


class RlSampleArgs(ctypes.Structure):
    _fields_ = [("logits", _P), ("N", _I64), ("V", _I64), ("row_stride", _I64), ("dtype", _I32), ("K", _I32),
                ("temperature", _P), ("top_k", _P), ("top_p", _P), ("min_p", _P), ("u", _P), ("tokens", _P),
                ("logq", _P), ("offsets", _P), ("ids", _P), ("support_logq", _P), ("capacity", _I64),
                ("replayed", _P)]


SIGS = {
    "rl_page_plan": (ctypes.c_int, [_P, _P, _P]),
    "rl_kv_append": (ctypes.c_int, [_P, _P, _P]),
    "rl_prefix_attn_workspace_bytes": (ctypes.c_size_t, [_P]),
    "rl_prefix_attn": (ctypes.c_int, [_P, _P, ctypes.c_size_t, _P, _P]),
    "rl_sample_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I32]),
    "rl_sample": (ctypes.c_int, [_P, _P, ctypes.c_size_t, _P, _P]),
}


def _packer(cls):
    """The C struct's bytes from the field values (None: a null pointer), several times faster
    than filling the ctypes structure."""
    code = {_P: "P", _I64: "q", _I32: "i", _F: "f"}
    fmt = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_) + "0q")
    assert fmt.size == ctypes.sizeof(cls)
    return fmt.pack


_pack_plan, _pack_append, _pack_attn, _pack_sample = (
    _packer(c) for c in (RlPagePlanArgs, RlKvAppendArgs, RlPrefixAttnArgs, RlSampleArgs))


def _err(msg):
    return sys.modules["lm_head_gb300"].RLHeadError(msg)


_lib = None
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _load():
    global _lib
    if _lib is None:
        _lib = sys.modules["lm_head_gb300"].load()
    return _lib


def _stream(stream, t):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(rc):
    if rc:
        sys.modules["lm_head_gb300"]._check(rc)


def _dev(name, t, dtype, n=None, optional=False):
    """Device address of a contiguous tensor of `dtype` (and `n` elements); 0 for none."""
    if t is None:
        if optional:
            return 0
        raise _err(f"{name} is missing")
    if not t.is_cuda:
        raise _err(f"{name}: librlhead takes device tensors; got a CPU tensor")
    if t.dtype is not dtype or not t.is_contiguous():
        raise _err(f"{name}: expected contiguous {dtype}, got {t.dtype}")
    if n is not None and t.numel() != n:
        raise _err(f"{name}: expected {n} elements, got {t.numel()}")
    return t.data_ptr()


def _on(stream):
    """What a call makes is made on the stream that the call runs on: a buffer zeroed on another one
    could be zeroed beside or after the call, and its memory be another's before the call is done."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _status(status, device):
    return torch.zeros(1, dtype=torch.int32, device=device) if status is None else status


@dataclasses.dataclass
class PagePlan:
    """What rl_page_plan writes (include/rlhead.h, rl_page_plan_args)."""
    cu_q: torch.Tensor          # [R+1] int32
    kv_lens: torch.Tensor       # [R] int32
    slot_map: torch.Tensor      # [T] int64
    positions: torch.Tensor     # [T] int32
    free_used: torch.Tensor     # [1] int32: pass it as the next step's free_used
    status: torch.Tensor        # [1] int32

    def status_bits(self) -> int:
        return int(self.status.item())


def rl_page_plan(q_lens, ctx_lens, block_table, free_pages, *, page_size: int, n_pages: int, n_tokens: int,
                 free_used=None, group_offsets=None, prefix_lens=None, out: Optional[PagePlan] = None, status=None,
                 stream=None) -> PagePlan:
    """Pages for a step's tokens: extends `block_table` [R, W] in place from the pool
    `free_pages` and returns the token offsets, key lengths, cache slots and positions.
    n_tokens is sum(q_lens), known to whoever sized the step's tensors.  out.free_used is another
    tensor than free_used; out.kv_lens may be ctx_lens."""
    R, W = block_table.shape
    i32 = torch.int32
    if out is None:
        dev = block_table.device
        if not block_table.is_cuda:
            raise _err("block_table: librlhead takes device tensors; got a CPU tensor")
        with _on(stream):
            out = PagePlan(torch.empty(R + 1, dtype=i32, device=dev), torch.empty(R, dtype=i32, device=dev),
                           torch.empty(n_tokens, dtype=torch.int64, device=dev),
                           torch.empty(n_tokens, dtype=i32, device=dev), torch.empty(1, dtype=i32, device=dev),
                           _status(status, dev))
    elif status is not None:
        out = dataclasses.replace(out, status=status)
    G = 0 if group_offsets is None else group_offsets.numel() - 1
    a = _pack_plan(R, n_tokens, _dev("q_lens", q_lens, i32, R), _dev("ctx_lens", ctx_lens, i32, R),
                       _dev("block_table", block_table, i32), W, _dev("free_pages", free_pages, i32),
                       free_pages.numel(), _dev("free_used", free_used, i32, 1, True),
                       _dev("out.free_used", out.free_used, i32, 1),
                       _dev("group_offsets", group_offsets, i32, None, True),
                       _dev("prefix_lens", prefix_lens, i32, G, G == 0), G, n_pages, page_size,
                       _dev("out.cu_q", out.cu_q, i32, R + 1), _dev("out.kv_lens", out.kv_lens, i32, R),
                       _dev("out.slot_map", out.slot_map, torch.int64, n_tokens),
                       _dev("out.positions", out.positions, i32, n_tokens, True))
    _check(_load().rl_page_plan(a, _dev("status", out.status, i32, 1), _stream(stream, block_table)))
    return out


def _cache(k_cache, v_cache):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise _err("k_cache / v_cache: two tensors [n_pages, Hkv, page_size, D] of one type")
    dt = k_cache.dtype
    return _dev("k_cache", k_cache, dt), _dev("v_cache", v_cache, dt), _DTYPES.get(dt, -1)


def rl_kv_append(k, v, slot_map, k_cache, v_cache, *, status=None, stream=None) -> torch.Tensor:
    """k_cache[slot] = k[t], v_cache[slot] = v[t] (k, v [T, Hkv, D], any token and head
    strides) for the tokens whose slot is not negative.  Returns the status word."""
    kc, vc, dt = _cache(k_cache, v_cache)
    n_pages, Hkv, page, D = k_cache.shape
    T = slot_map.numel()
    for name, t in (("k", k), ("v", v)):
        if not t.is_cuda or t.dtype != k_cache.dtype or tuple(t.shape) != (T, Hkv, D) or (D > 1 and t.stride(2) != 1):
            raise _err(f"{name}: expected a device tensor [{T}, {Hkv}, {D}] of the cache's type with dense heads")
    if status is None:
        with _on(stream):
            status = _status(None, k_cache.device)
    a = _pack_append(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                       _dev("slot_map", slot_map, torch.int64, T), kc, vc, T, n_pages, Hkv, D, page, dt)
    _check(_load().rl_kv_append(a, _dev("status", status, torch.int32, 1), _stream(stream, k_cache)))
    return status


@dataclasses.dataclass
class AttnOut:
    out: torch.Tensor           # [T, Hq, D], the cache's type
    lse: Optional[torch.Tensor]  # [T, Hq] fp32
    ws: torch.Tensor
    status: torch.Tensor

    def status_bits(self) -> int:
        return int(self.status.item())


def rl_prefix_attn(q, k_cache, v_cache, cu_q, kv_lens, block_table, *, max_q: int, max_kv: int, group_offsets=None,
                   prefix_lens=None, prefix_table=None, max_prefix: Optional[int] = None, scale: Optional[float] = None,
                   out: Optional[AttnOut] = None, ws=None, status=None, stream=None) -> AttnOut:
    """Attention of a step's queries q [T, Hq, D] (any token and head strides) over their
    group's shared prefix and each request's own keys, causal within the step.  max_q, max_kv
    and max_prefix bound the device lengths (max_prefix: what prefix_table has room for, by
    default).  scale: 1 / sqrt(D) by default."""
    kc, vc, dt = _cache(k_cache, v_cache)
    n_pages, Hkv, page, D = k_cache.shape
    if not q.is_cuda or q.dim() != 3 or q.dtype != k_cache.dtype or q.shape[2] != D or q.stride(2) != 1:
        raise _err(f"q: expected a device tensor [T, Hq, {D}] of the cache's type with dense heads")
    T, Hq, _ = q.shape
    i32 = torch.int32
    R, W = block_table.shape
    G = 0 if group_offsets is None else group_offsets.numel() - 1
    WP = 0
    if G:
        if prefix_table is None or prefix_table.dim() != 2 or prefix_table.shape[0] != G:
            raise _err(f"prefix_table: expected [{G}, pages]")
        WP = prefix_table.shape[1]
    if max_prefix is None:
        max_prefix = WP * page
    head = (q.data_ptr(), q.stride(0), q.stride(1), kc, vc, n_pages, T, R, G, _dev("cu_q", cu_q, i32, R + 1),
            _dev("kv_lens", kv_lens, i32, R), _dev("block_table", block_table, i32), W,
            _dev("group_offsets", group_offsets, i32, None, True), _dev("prefix_lens", prefix_lens, i32, G, G == 0),
            _dev("prefix_table", prefix_table, i32, None, G == 0), WP, max_q, max_kv, max_prefix, Hq, Hkv, D, page, dt,
            D ** -0.5 if scale is None else scale)
    if out is None:
        dev = q.device
        with _on(stream):
            if ws is None:
                n = int(_load().rl_prefix_attn_workspace_bytes(_pack_attn(*head, 0, 0)))
                ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
            out = AttnOut(torch.empty(T, Hq, D, dtype=q.dtype, device=dev),
                          torch.empty(T, Hq, dtype=torch.float32, device=dev), ws, _status(status, dev))
    elif status is not None or ws is not None:
        out = dataclasses.replace(out, status=out.status if status is None else status, ws=out.ws if ws is None else ws)
    a = _pack_attn(*head, _dev("out.out", out.out, q.dtype, T * Hq * D),
                   _dev("out.lse", out.lse, torch.float32, T * Hq, True))
    _check(_load().rl_prefix_attn(a, _dev("ws", out.ws, torch.uint8), out.ws.numel(),
                                  _dev("status", out.status, i32, 1), _stream(stream, q)))
    return out


@dataclasses.dataclass
class SampleOut:
    """What rl_sample writes (include/rlhead.h, rl_sample_args).  The support rows are the
    head's CSR: HeadBatch takes offsets, ids[:nnz], support_logq[:nnz] and replayed as they are."""
    tokens: torch.Tensor                     # [N, K] int32
    logq: torch.Tensor                       # [N, K] fp32
    offsets: Optional[torch.Tensor]          # [N+1] int64
    ids: Optional[torch.Tensor]              # [capacity] int32
    support_logq: Optional[torch.Tensor]     # [capacity] fp32
    replayed: torch.Tensor                   # [N] uint8
    ws: torch.Tensor
    status: torch.Tensor

    def status_bits(self) -> int:
        return int(self.status.item())

    def nnz(self) -> int:
        """Support entries (a device read): more than the buffers hold if CAPACITY is set."""
        return int(self.offsets[-1].item())


def rl_sample_workspace_bytes(N: int, V: int, K: int) -> int:
    return int(_load().rl_sample_workspace_bytes(N, V, K))


def rl_sample(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, capacity: int = 0,
              out: Optional[SampleOut] = None, ws=None, status=None, stream=None) -> SampleOut:
    """K draws a row (u [N, K] in [0, 1)) from logits [N, V] (fp32, bf16 or fp16; any row
    stride) under each row's temperature, top-k, top-p and min-p ([N] tensors or None), with
    the log-probability of each draw under the truncated distribution.  capacity > 0 also
    writes the sampler support rows, up to that many entries."""
    f32, i32 = torch.float32, torch.int32
    if not logits.is_cuda or logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise _err("logits: expected a device tensor [N, V] with dense rows")
    N, V = logits.shape
    if u.dim() != 2 or u.shape[0] != N:
        raise _err(f"u: expected [{N}, K]")
    K = u.shape[1]
    if out is None:
        dev = logits.device
        e = lambda n, dt: torch.empty(n, dtype=dt, device=dev)  # noqa: E731
        with _on(stream):
            if ws is None:
                ws = torch.empty(max(rl_sample_workspace_bytes(N, V, K), 1), dtype=torch.uint8, device=dev)
            out = SampleOut(e((N, K), i32), e((N, K), f32), e(N + 1, torch.int64) if capacity else None,
                            torch.zeros(capacity, dtype=i32, device=dev) if capacity else None,
                            torch.zeros(capacity, dtype=f32, device=dev) if capacity else None, e(N, torch.uint8), ws,
                            _status(status, dev))
    elif status is not None or ws is not None:
        out = dataclasses.replace(out, status=out.status if status is None else status, ws=out.ws if ws is None else ws)
    a = _pack_sample(logits.data_ptr(), N, V, logits.stride(0) if N > 1 else V, _DTYPES.get(logits.dtype, -1), K,
                     _dev("temperature", temperature, f32, N, True), _dev("top_k", top_k, i32, N, True),
                     _dev("top_p", top_p, f32, N, True), _dev("min_p", min_p, f32, N, True), _dev("u", u, f32, N * K),
                     _dev("out.tokens", out.tokens, i32, N * K), _dev("out.logq", out.logq, f32, N * K, True),
                     _dev("out.offsets", out.offsets, torch.int64, N + 1, True),
                     _dev("out.ids", out.ids, i32, capacity, True),
                     _dev("out.support_logq", out.support_logq, f32, capacity, True), capacity,
                     _dev("out.replayed", out.replayed, torch.uint8, N, True))
    _check(_load().rl_sample(a, _dev("ws", out.ws, torch.uint8), out.ws.numel(), _dev("status", out.status, i32, 1),
                             _stream(stream, logits)))
    return out
