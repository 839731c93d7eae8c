"""Binding of the distillation calls (include/rlhead.h, "distillation from a teacher's top tokens")."""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Union

import torch

from .generation import _DTYPES, _F, _I32, _I64, _P, _check, _dev, _err, _load, _on, _packer, _status, _stream

RL_DISTILL_FORWARD, RL_DISTILL_REVERSE, RL_DISTILL_JSD = 0, 1, 2
_KINDS = {"forward": RL_DISTILL_FORWARD, "reverse": RL_DISTILL_REVERSE, "jsd": RL_DISTILL_JSD}


class RlDistillArgs(ctypes.Structure):
    _fields_ = [("logits", _P), ("N", _I64), ("V", _I64), ("row_stride", _I64), ("dtype", _I32), ("kind", _I32), ("tail", _I32),
                ("temperature", _F), ("beta", _F), ("reserved", _I32), ("offsets", _P), ("ids", _P), ("logq", _P), ("nnz", _I64),
                ("dloss", _P), ("dlogits", _P), ("grad_stride", _I64), ("loss", _P), ("mass", _P)]


SIGS = {
    "rl_distill_saved_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "rl_distill_fwd": (ctypes.c_int, [_P, _P, _P, _P]),
    "rl_distill_bwd": (ctypes.c_int, [_P, _P, _P, _P]),
    "rl_distill_fwd_bwd": (ctypes.c_int, [_P, _P, _P, _P]),
}
_pack = _packer(RlDistillArgs)


@dataclasses.dataclass
class DistillParams:
    """kind: "forward" (KL of the student from the teacher), "reverse" or "jsd".  tail: the rest of the
    vocabulary is one more outcome (the other kinds need it)."""
    kind: Union[str, int] = "forward"
    tail: bool = False
    temperature: float = 1.0
    beta: float = 0.5


@dataclasses.dataclass
class DistillOut:
    loss: torch.Tensor              # [N] fp32
    mass: torch.Tensor              # [N] fp32: the student's probability of the support
    saved: torch.Tensor             # workspace; what the forward leaves for the backward
    status: torch.Tensor

    def status_bits(self) -> int:
        return int(self.status.item())


def _head(logits, offsets, ids, logq, p):
    if not logits.is_cuda or logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1) or logits.dtype not in _DTYPES:
        raise _err("logits: expected a device tensor [N, V] (fp32, bf16 or fp16) with dense rows")
    N, V = logits.shape
    kind = _KINDS.get(p.kind, -1) if isinstance(p.kind, str) else p.kind
    nnz = ids.numel()
    return (logits.data_ptr(), N, V, logits.stride(0) if N > 1 else V, _DTYPES[logits.dtype], kind, int(p.tail),
            p.temperature, p.beta, 0, _dev("offsets", offsets, torch.int64, N + 1), _dev("ids", ids, torch.int32),
            _dev("logq", logq, torch.float32, nnz), nnz)


def _outputs(logits, nnz, out, status, stream):
    N = logits.shape[0]
    n = int(_load().rl_distill_saved_bytes(N, nnz))
    if out is None:
        with _on(stream):
            dev = logits.device
            e = lambda k, t: torch.empty(k, dtype=t, device=dev)  # noqa: E731
            return DistillOut(e(N, torch.float32), e(N, torch.float32), e(max(n, 1), torch.uint8), _status(status, dev))
    if out.saved.numel() < n:
        raise _err(f"out.saved: expected {n} bytes")
    return out if status is None else dataclasses.replace(out, status=status)


def _grad(logits, dlogits, stream):
    if dlogits is None:
        with _on(stream):
            return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype or not dlogits.is_cuda or \
            (logits.shape[1] > 1 and dlogits.stride(1) != 1):
        raise _err("dlogits: expected a device tensor like logits, with dense rows")
    return dlogits


def _tail_args(o, N):
    f32 = torch.float32
    return _dev("out.loss", o.loss, f32, N), _dev("out.mass", o.mass, f32, N, True)


def rl_distill_fwd(logits, offsets, ids, logq, params: DistillParams, *, out: Optional[DistillOut] = None, status=None,
                   stream=None) -> DistillOut:
    """The loss of each row of `logits` [N, V] against its support row of a teacher (offsets [N+1] int64, ids int32
    ascending, logq fp32), and what rl_distill_bwd needs (out.saved)."""
    head = _head(logits, offsets, ids, logq, params)
    out = _outputs(logits, ids.numel(), out, status, stream)
    a = _pack(*head, 0, 0, 0, *_tail_args(out, logits.shape[0]))
    _check(_load().rl_distill_fwd(a, _dev("out.saved", out.saved, torch.uint8), _dev("status", out.status, torch.int32, 1),
                                  _stream(stream, logits)))
    return out


def rl_distill_bwd(logits, offsets, ids, logq, params: DistillParams, saved, dloss, *, dlogits=None, status=None, stream=None):
    """Gradients [N, V] for the rows' dloss [N] from what the forward saved; dlogits may be logits.  Returns (dlogits, status)."""
    head = _head(logits, offsets, ids, logq, params)
    N = logits.shape[0]
    if saved is None or saved.numel() < int(_load().rl_distill_saved_bytes(N, ids.numel())):
        raise _err("saved: expected what rl_distill_fwd left for these rows")
    d = _grad(logits, dlogits, stream)
    if status is None:
        with _on(stream):
            status = _status(None, logits.device)
    a = _pack(*head, _dev("dloss", dloss, torch.float32, N), d.data_ptr(), d.stride(0) if N > 1 else logits.shape[1], 0, 0)
    _check(_load().rl_distill_bwd(a, _dev("saved", saved, torch.uint8), _dev("status", status, torch.int32, 1),
                                  _stream(stream, logits)))
    return d, status


def rl_distill_fwd_bwd(logits, offsets, ids, logq, dloss, params: DistillParams, *, out: Optional[DistillOut] = None, dlogits=None,
                       status=None, stream=None):
    """Loss and gradients in one pass over the logits; dlogits may be logits.  Returns (out, dlogits)."""
    head = _head(logits, offsets, ids, logq, params)
    N = logits.shape[0]
    out = _outputs(logits, ids.numel(), out, status, stream)
    d = _grad(logits, dlogits, stream)
    a = _pack(*head, _dev("dloss", dloss, torch.float32, N), d.data_ptr(), d.stride(0) if N > 1 else logits.shape[1],
              *_tail_args(out, N))
    _check(_load().rl_distill_fwd_bwd(a, _dev("out.saved", out.saved, torch.uint8), _dev("status", out.status, torch.int32, 1),
                                      _stream(stream, logits)))
    return out, d
