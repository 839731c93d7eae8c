"""Binding of the verification of drafted tokens (include/rlhead.h, rl_verify)."""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from .generation import _DTYPES, _I32, _I64, _P, _check, _dev, _err, _load, _on, _packer, _status, _stream

_DIST = [("logits", _P), ("n_rows", _I64), ("row_stride", _I64), ("temperature", _P), ("offsets", _P), ("ids", _P), ("logq", _P),
         ("nnz", _I64), ("replayed", _P), ("rows", _P)]


class RlVerifyArgs(ctypes.Structure):
    # (the two rl_dist in line)
    _fields_ = [("R", _I64), ("T", _I64), ("V", _I64), ("cu_q", _P), ("step_tokens", _P), ("u", _P), ("u_next", _P)] + \
        [("target_" + n, t) for n, t in _DIST] + [("draft_" + n, t) for n, t in _DIST] + \
        [("target_dtype", _I32), ("draft_dtype", _I32), ("ctx_lens", _P), ("tokens", _P), ("logq", _P), ("accepted", _P),
         ("keep_lens", _P)]


SIGS = {
    "rl_verify_workspace_bytes": (ctypes.c_size_t, [_P]),
    "rl_verify": (ctypes.c_int, [_P, _P, ctypes.c_size_t, _P, _P]),
}
_pack = _packer(RlVerifyArgs)


@dataclasses.dataclass
class Dist:
    """The distributions of rows: logits [n, V] with temperatures [n], support rows as rl_sample writes them (offsets [n+1], ids,
    logq), or both, each row by replayed [n].  rows [T]: which of them the step's row t has (t by default)."""
    logits: Optional[torch.Tensor] = None
    temperature: Optional[torch.Tensor] = None
    offsets: Optional[torch.Tensor] = None
    ids: Optional[torch.Tensor] = None
    logq: Optional[torch.Tensor] = None
    replayed: Optional[torch.Tensor] = None
    rows: Optional[torch.Tensor] = None


@dataclasses.dataclass
class VerifyOut:
    tokens: torch.Tensor                # [T] int32: accepted tokens, the new one, then -1
    logq: torch.Tensor                  # [T] fp32: ln p of each under the target
    accepted: torch.Tensor              # [R] int32
    keep_lens: torch.Tensor             # [R] int32: for rl_page_release
    ws: torch.Tensor
    status: torch.Tensor

    def status_bits(self) -> int:
        return int(self.status.item())


_NONE = (0,) * len(_DIST)


def _dist(name, d, V, T):
    """(fields of rl_dist, dtype code)."""
    if d is None:
        return _NONE, 0
    f32, i32 = torch.float32, torch.int32
    z, dt, stride, n = d.logits, 0, 0, None
    if z is not None:
        if not z.is_cuda or z.dim() != 2 or z.shape[1] != V or z.dtype not in _DTYPES or (V > 1 and z.stride(1) != 1):
            raise _err(f"{name}.logits: expected a device tensor [rows, {V}] (fp32, bf16 or fp16) with dense rows")
        n, dt = z.shape[0], _DTYPES[z.dtype]
        stride = z.stride(0) if n > 1 else V
    if d.offsets is not None:
        m = d.offsets.numel() - 1
        if n is not None and m != n:
            raise _err(f"{name}.offsets: expected {n + 1} elements, got {m + 1}")
        n = m
    if n is None:
        raise _err(f"{name}: neither logits nor support rows")
    if d.rows is None and n < T:
        raise _err(f"{name}: {n} rows for a step of {T}")
    has = d.offsets is not None
    nnz = d.ids.numel() if has and d.ids is not None else 0
    # (no rows have no address, and a null one would say that there are no logits at all; nothing of it is read)
    at = 0 if z is None else z.data_ptr() or 16
    return (at, n, stride, _dev(f"{name}.temperature", d.temperature, f32, n, True),
            _dev(f"{name}.offsets", d.offsets, torch.int64, None, True), _dev(f"{name}.ids", d.ids, i32, None, not has),
            _dev(f"{name}.logq", d.logq, f32, nnz, not has), nnz, _dev(f"{name}.replayed", d.replayed, torch.uint8, n, True),
            _dev(f"{name}.rows", d.rows, i32, T, True)), dt


def rl_verify(step_tokens, cu_q, u, u_next, target: Dist, draft: Optional[Dist] = None, *, vocab: int, ctx_lens=None,
              out: Optional[VerifyOut] = None, ws=None, status=None, stream=None) -> VerifyOut:
    """Which drafted tokens the target accepts, and the token after them.  The step's tokens [T] are each request's last
    token and its drafts (rows cu_q[r] .. cu_q[r+1], as rl_page_plan wrote them); row t of `target` is the target's distribution after
    token t, row t of `draft` the one that token t + 1 was drafted from (None: the drafts were certain).  u [T] and u_next [R]
    are random numbers in [0, 1)."""
    i32, f32 = torch.int32, torch.float32
    T, R = step_tokens.numel(), u_next.numel()
    td, tt = _dist("target", target, vocab, T)
    if target is None:
        raise _err("target is missing")
    dd, dt = _dist("draft", draft, vocab, T)
    head = (R, T, vocab, _dev("cu_q", cu_q, i32, R + 1), _dev("step_tokens", step_tokens, i32), _dev("u", u, f32, T),
            _dev("u_next", u_next, f32, R), *td, *dd, tt, dt, _dev("ctx_lens", ctx_lens, i32, R, True))
    if out is None:
        dev = step_tokens.device
        with _on(stream):
            e = lambda n, t: torch.empty(n, dtype=t, device=dev)  # noqa: E731
            if ws is None:
                ws = e(max(int(_load().rl_verify_workspace_bytes(_pack(*head, 0, 0, 0, 0))), 1), torch.uint8)
            out = VerifyOut(e(T, i32), e(T, f32), e(R, i32), e(R, i32), ws, _status(status, dev))
    elif status is not None or ws is not None:
        out = dataclasses.replace(out, status=out.status if status is None else status, ws=out.ws if ws is None else ws)
    a = _pack(*head, _dev("out.tokens", out.tokens, i32, T), _dev("out.logq", out.logq, f32, T, True),
              _dev("out.accepted", out.accepted, i32, R), _dev("out.keep_lens", out.keep_lens, i32, R, True))
    _check(_load().rl_verify(a, _dev("ws", out.ws, torch.uint8), out.ws.numel(), _dev("status", out.status, i32, 1),
                             _stream(stream, step_tokens)))
    return out
