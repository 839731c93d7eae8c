"""Binding of the calls that give back, share, copy and move pages of a cache (include/rlhead.h,
"several tokens a step, and the pages of a rollout's life").

As in the generation module: argument marshalling only, outputs through `out` / `status`, so
that a loop allocates nothing after its first step and can be captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from .generation import _DTYPES, _I32, _I64, _P, _check, _dev, _err, _load, _on, _packer, _status, _stream


class RlPageReleaseArgs(ctypes.Structure):
    _fields_ = [("R", _I64), ("kv_lens", _P), ("keep_lens", _P), ("block_table", _P), ("table_width", _I64), ("G", _I64),
                ("held_lens", _P), ("held_table", _P), ("held_width", _I64), ("free_pages", _P), ("n_free", _I64),
                ("free_used", _P), ("free_used_out", _P), ("n_pages", _I64), ("page_size", _I32)]


class RlPageForkArgs(ctypes.Structure):
    _fields_ = [("R", _I64), ("C", _I64), ("parents", _P), ("children", _P), ("lens", _P), ("kv_lens", _P),
                ("block_table", _P), ("table_width", _I64), ("free_pages", _P), ("n_free", _I64), ("free_used", _P),
                ("free_used_out", _P), ("n_pages", _I64), ("src", _P), ("dst", _P), ("tokens", _P), ("page_size", _I32)]


class RlPageCompactArgs(ctypes.Structure):
    _fields_ = [("R", _I64), ("kv_lens", _P), ("block_table", _P), ("block_table_out", _P), ("table_width", _I64), ("G", _I64),
                ("prefix_lens", _P), ("prefix_table", _P), ("prefix_table_out", _P), ("prefix_width", _I64), ("n_pages", _I64),
                ("src", _P), ("dst", _P), ("free_pages", _P), ("free_used_out", _P), ("page_size", _I32)]


class RlPageCopyArgs(ctypes.Structure):
    _fields_ = [("n", _I64), ("src", _P), ("dst", _P), ("tokens", _P), ("k_cache", _P), ("v_cache", _P), ("layer_stride", _I64),
                ("n_pages", _I64), ("layers", _I32), ("Hkv", _I32), ("D", _I32), ("page_size", _I32), ("dtype", _I32)]


_SZ = ctypes.c_size_t
SIGS = {
    "rl_page_release_workspace_bytes": (_SZ, [_I64]),
    "rl_page_release": (ctypes.c_int, [_P, _P, _SZ, _P, _P]),
    "rl_page_fork_workspace_bytes": (_SZ, [_I64, _I64]),
    "rl_page_fork": (ctypes.c_int, [_P, _P, _SZ, _P, _P]),
    "rl_page_compact_workspace_bytes": (_SZ, [_I64]),
    "rl_page_compact": (ctypes.c_int, [_P, _P, _SZ, _P, _P]),
    "rl_page_copy": (ctypes.c_int, [_P, _P, _P]),
}
_pack_release, _pack_fork, _pack_compact, _pack_copy = (
    _packer(c) for c in (RlPageReleaseArgs, RlPageForkArgs, RlPageCompactArgs, RlPageCopyArgs))
_i32 = torch.int32


def _table(name, t, rows=None):
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows):
        raise _err(f"{name}: expected [{'rows' if rows is None else rows}, pages]")
    return _dev(name, t, _i32), t.shape[0], t.shape[1]


def _workspace(ws, nbytes, device):
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device) if ws is None else ws


def _given(out, ws, status):
    """`out` with the caller's own workspace and status word in place of its."""
    if ws is None and status is None:
        return out
    return dataclasses.replace(out, ws=out.ws if ws is None else ws, status=out.status if status is None else status)


class _Bits:
    def status_bits(self) -> int:
        return int(self.status.item())


@dataclasses.dataclass
class PageRelease(_Bits):
    free_used: torch.Tensor     # [1] int32: pass it as the next step's free_used
    ws: torch.Tensor
    status: torch.Tensor


def rl_page_release(kv_lens, keep_lens, block_table, free_pages, free_used, *, page_size: int, n_pages: int,
                    held_lens=None, held_table=None, out: Optional[PageRelease] = None, ws=None, status=None,
                    stream=None) -> PageRelease:
    """Gives the pages that no row needs any more back to the pool `free_pages` (in place).  Rows keep their
    first keep_lens tokens of kv_lens; the pages of the held rows all stay.  out.free_used is another tensor
    than free_used."""
    table, R, W = _table("block_table", block_table)
    G = 0 if held_lens is None else held_lens.numel()
    held, _, WG = _table("held_table", held_table, G) if G else (0, 0, 0)
    if out is None:
        with _on(stream):
            dev = block_table.device
            out = PageRelease(torch.empty(1, dtype=_i32, device=dev),
                              _workspace(ws, int(_load().rl_page_release_workspace_bytes(n_pages)), dev), _status(status, dev))
    else:
        out = _given(out, ws, status)
    a = _pack_release(R, _dev("kv_lens", kv_lens, _i32, R), _dev("keep_lens", keep_lens, _i32, R), table, W, G,
                      _dev("held_lens", held_lens, _i32, G, G == 0), held, WG, _dev("free_pages", free_pages, _i32),
                      free_pages.numel(), _dev("free_used", free_used, _i32, 1), _dev("out.free_used", out.free_used, _i32, 1),
                      n_pages, page_size)
    _check(_load().rl_page_release(a, _dev("ws", out.ws, torch.uint8), out.ws.numel(), _dev("status", out.status, _i32, 1),
                                   _stream(stream, block_table)))
    return out


@dataclasses.dataclass
class PageFork(_Bits):
    src: torch.Tensor           # [C] int32: the copies to make, for rl_page_copy
    dst: torch.Tensor           # [C] int32
    tokens: torch.Tensor        # [C] int32
    free_used: torch.Tensor     # [1] int32
    ws: torch.Tensor
    status: torch.Tensor


def rl_page_fork(parents, children, lens, kv_lens, block_table, free_pages, free_used, *, page_size: int, n_pages: int,
                 out: Optional[PageFork] = None, ws=None, status=None, stream=None) -> PageFork:
    """Row children[c] of `block_table` and `kv_lens` (both in place) goes on from the first lens[c] tokens of row
    parents[c], sharing its full pages.  Copy the last ones with rl_page_copy(out.src, out.dst, ..., tokens=out.tokens)
    in every layer's cache."""
    table, R, W = _table("block_table", block_table)
    C = parents.numel()
    if out is None:
        with _on(stream):
            dev = block_table.device
            e = lambda n: torch.empty(n, dtype=_i32, device=dev)  # noqa: E731
            out = PageFork(e(C), e(C), e(C), e(1), _workspace(ws, int(_load().rl_page_fork_workspace_bytes(R, C)), dev),
                           _status(status, dev))
    else:
        out = _given(out, ws, status)
    a = _pack_fork(R, C, _dev("parents", parents, _i32), _dev("children", children, _i32, C), _dev("lens", lens, _i32, C),
                   _dev("kv_lens", kv_lens, _i32, R), table, W, _dev("free_pages", free_pages, _i32), free_pages.numel(),
                   _dev("free_used", free_used, _i32, 1), _dev("out.free_used", out.free_used, _i32, 1), n_pages,
                   _dev("out.src", out.src, _i32, C), _dev("out.dst", out.dst, _i32, C),
                   _dev("out.tokens", out.tokens, _i32, C), page_size)
    _check(_load().rl_page_fork(a, _dev("ws", out.ws, torch.uint8), out.ws.numel(), _dev("status", out.status, _i32, 1),
                                _stream(stream, block_table)))
    return out


@dataclasses.dataclass
class PageCompact(_Bits):
    block_table: torch.Tensor              # [R, W] int32, with the new ids
    prefix_table: Optional[torch.Tensor]   # [G, WP] int32
    src: torch.Tensor                      # [n_pages / 2] int32: the moves to make, for rl_page_copy
    dst: torch.Tensor                      # [n_pages / 2] int32
    free_pages: torch.Tensor               # [n_pages] int32
    free_used: torch.Tensor                # [1] int32: the number of live pages
    ws: torch.Tensor
    status: torch.Tensor


def rl_page_compact(kv_lens, block_table, *, page_size: int, n_pages: int, prefix_lens=None, prefix_table=None,
                    out: Optional[PageCompact] = None, ws=None, status=None, stream=None) -> PageCompact:
    """New tables in which the live pages have the ids 0 .. n_live - 1, the moves that take their contents there
    (rl_page_copy(out.src, out.dst, ...) in every layer's cache), and the pool to go on with.  A table of `out` may be
    the one given."""
    table, R, W = _table("block_table", block_table)
    G = 0 if prefix_lens is None else prefix_lens.numel()
    prefix, _, WP = _table("prefix_table", prefix_table, G) if G else (0, 0, 0)
    if out is None:
        with _on(stream):
            dev = block_table.device
            e = lambda *n: torch.empty(n, dtype=_i32, device=dev)  # noqa: E731
            out = PageCompact(e(R, W), e(G, WP) if G else None, e(n_pages // 2), e(n_pages // 2), e(n_pages), e(1),
                              _workspace(ws, int(_load().rl_page_compact_workspace_bytes(n_pages)), dev), _status(status, dev))
    else:
        out = _given(out, ws, status)
    half = n_pages // 2
    a = _pack_compact(R, _dev("kv_lens", kv_lens, _i32, R), table, _dev("out.block_table", out.block_table, _i32, R * W), W, G,
                      _dev("prefix_lens", prefix_lens, _i32, G, G == 0), prefix,
                      _dev("out.prefix_table", out.prefix_table, _i32, G * WP) if G else 0, WP, n_pages,
                      _dev("out.src", out.src, _i32, half), _dev("out.dst", out.dst, _i32, half),
                      _dev("out.free_pages", out.free_pages, _i32, n_pages), _dev("out.free_used", out.free_used, _i32, 1),
                      page_size)
    _check(_load().rl_page_compact(a, _dev("ws", out.ws, torch.uint8), out.ws.numel(), _dev("status", out.status, _i32, 1),
                                   _stream(stream, block_table)))
    return out


def rl_page_copy(src, dst, k_cache, v_cache, *, tokens=None, status=None, stream=None) -> torch.Tensor:
    """Page dst[i] of the caches = page src[i] (its first tokens[i] tokens, or all).  The caches: [n_pages, Hkv, page_size, D],
    or [layers, n_pages, Hkv, page_size, D] with each layer dense.  Returns the status word."""
    shape, dt = k_cache.shape, k_cache.dtype
    if k_cache.dim() not in (4, 5) or v_cache.shape != shape or v_cache.dtype != dt or dt not in _DTYPES:
        raise _err("k_cache / v_cache: two tensors [layers, n_pages, Hkv, page_size, D] of one type")
    many = k_cache.dim() == 5
    layers, stride = (shape[0], k_cache.stride(0)) if many else (1, 0)
    dense = k_cache.is_contiguous() and v_cache.is_contiguous()
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_cuda:
            raise _err(f"{name}: librlhead takes device tensors; got a CPU tensor")
        if dense:
            continue
        one = t[0] if many and layers else t
        if not one.is_contiguous() or (many and layers > 1 and t.stride(0) != stride):
            raise _err(f"{name}: expected dense layers, as far apart in both caches")
    n_pages, Hkv, page, D = shape[-4:]
    n = src.numel()
    if status is None:
        with _on(stream):
            status = _status(None, k_cache.device)
    a = _pack_copy(n, _dev("src", src, _i32), _dev("dst", dst, _i32, n), _dev("tokens", tokens, _i32, n, True),
                   k_cache.data_ptr(), v_cache.data_ptr(), stride, n_pages, layers, Hkv, D, page, _DTYPES[dt])
    _check(_load().rl_page_copy(a, _dev("status", status, _i32, 1), _stream(stream, k_cache)))
    return status
