"""Distillation, host side: what is refused before any device work."""
import ctypes

import pytest
import torch

import lm_head_gb300 as rh
from lm_head_gb300 import distill as ds
from test_generation_cpu import FAKE, _fill, lib  # noqa: F401

ARG, UNS = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED


def make(**kw):
    far = FAKE + (1 << 30)
    return _fill(ds.RlDistillArgs, **{**dict(N=4, V=1000, row_stride=1000, dtype=rh.RL_DTYPE_F32, kind=1, tail=1, temperature=1.0,
                                             beta=0.5, reserved=0, nnz=10, grad_stride=1000, dlogits=far), **kw})


COMMON = [
    (dict(N=-1), ARG), (dict(V=0), ARG), (dict(nnz=-1), ARG), (dict(dtype=3), UNS), (dict(kind=3), ARG), (dict(kind=-1), ARG),
    (dict(tail=2), ARG), (dict(tail=0), ARG), (dict(tail=0, kind=2), ARG), (dict(reserved=1), ARG), (dict(temperature=0.0), ARG),
    (dict(temperature=-1.0), ARG), (dict(temperature=float("nan")), ARG), (dict(temperature=float("inf")), ARG),
    (dict(temperature=2.0 ** 21), ARG), (dict(kind=2, beta=0.0), ARG), (dict(kind=2, beta=1.0), ARG),
    (dict(kind=2, beta=float("nan")), ARG), (dict(V=450001, row_stride=450001, grad_stride=450001), UNS), (dict(N=1 << 31), UNS),
    (dict(row_stride=999), ARG), (dict(logits=None), ARG), (dict(offsets=None), ARG), (dict(ids=None), ARG), (dict(logq=None), ARG),
    (dict(logits=FAKE + 2), ARG)]
GRAD = [(dict(dloss=None), ARG), (dict(dlogits=None), ARG), (dict(dlogits=FAKE + (1 << 30) + 2), ARG), (dict(grad_stride=999), ARG),
        (dict(dlogits=FAKE + 4), ARG), (dict(dlogits=FAKE, grad_stride=1001), ARG), (dict(dlogits=FAKE + 4 * 3999), ARG)]


def test_refusals(lib):  # noqa: F811
    for changes, call in (
            (COMMON + [(dict(loss=None), ARG)], lambda a: lib.rl_distill_fwd(a, FAKE, FAKE, None)),
            (COMMON + GRAD, lambda a: lib.rl_distill_bwd(a, FAKE, FAKE, None)),
            (COMMON + GRAD + [(dict(loss=None), ARG)], lambda a: lib.rl_distill_fwd_bwd(a, FAKE, FAKE, None))):
        for change, want in changes:
            assert call(ctypes.byref(make(**change))) == want, change
        assert call(None) == ARG
    a = ctypes.byref(make())
    assert lib.rl_distill_fwd(a, FAKE, None, None) == ARG                # no status word
    assert lib.rl_distill_bwd(a, None, FAKE, None) == ARG                # nothing saved
    assert lib.rl_distill_fwd(a, FAKE + 8, FAKE, None) == ARG and lib.rl_distill_fwd(a, None, FAKE, None) == ARG
    assert lib.rl_distill_fwd_bwd(a, None, FAKE, None) == ARG
    assert rh.load().rl_distill_saved_bytes(-1, 0) == 0 and rh.load().rl_distill_saved_bytes(10, 20) >= 4 * 70
    assert ctypes.sizeof(ds.RlDistillArgs) == 4 * 8 + 6 * 4 + 9 * 8


def test_binding_refuses_wrong_tensors():
    z, e = torch.zeros(2, 10), torch.zeros(3)
    off, ids = torch.tensor([0, 1, 3]), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(rh.RLHeadError):
        rh.rl_distill_fwd(z, off, ids, e, rh.DistillParams())
    with pytest.raises(rh.RLHeadError):
        rh.rl_distill_fwd_bwd(z.to(torch.int32), off, ids, e, torch.ones(2), rh.DistillParams())


def test_gradients_between_the_rows_of_the_logits(lib):  # noqa: F811
    """Halves of one buffer share no memory, whatever their ranges; anything that does is refused."""
    def call(**kw):
        a = make(row_stride=2000, grad_stride=2000, **kw)
        return lib.rl_distill_bwd(ctypes.byref(a), FAKE + (1 << 28), FAKE, None)
    if not torch.cuda.is_available():
        for d in (1000, -1000, 1000 - 2 * 2000, 1000 + 3 * 2000):
            assert call(dlogits=FAKE + 4 * d) not in (rh.RL_OK, ARG), d         # (no device)
        assert call(dlogits=FAKE + 4 * 1000, N=1) not in (rh.RL_OK, ARG)
    for d in (999, 1001, -999, -1001, 2000, 1, 4001, -2000):
        assert call(dlogits=FAKE + 4 * d) == ARG, d
    a = make(row_stride=2000, grad_stride=3000, dlogits=FAKE + 4000)             # (other strides: some rows do)
    assert lib.rl_distill_bwd(ctypes.byref(a), FAKE + (1 << 28), FAKE, None) == ARG


def test_outputs_that_share_memory(lib):  # noqa: F811
    """Each input's first and last element under each output; the loss in dloss's place is sound."""
    size = dict(logits=16000, offsets=40, ids=40, logq=40, dloss=16, loss=16, mass=16, dlogits=16000)
    apart = {n: FAKE + (k << 16) for k, n in enumerate(size)}
    state = FAKE + (1 << 28)
    calls = dict(fwd=lib.rl_distill_fwd, bwd=lib.rl_distill_bwd, fwd_bwd=lib.rl_distill_fwd_bwd)
    outs = dict(fwd=("loss", "mass"), bwd=("dlogits",), fwd_bwd=("loss", "mass", "dlogits"))

    def call(name, saved=state, **kw):
        a = make(**{**apart, **kw})
        return calls[name](ctypes.byref(a), saved, FAKE + (1 << 27), None)
    for name, fn in calls.items():
        ins = ["logits", "offsets", "ids", "logq"] + (["dloss"] if name != "fwd" else [])
        for x in ins:
            for y in outs[name]:
                if (x, y) in (("logits", "dlogits"), ("dloss", "loss"), ("dloss", "mass")):
                    continue
                assert call(name, **{y: apart[x]}) == call(name, **{y: apart[x] + size[x] - 4}) == ARG, (name, x, y)
            assert call(name, saved=apart[x]) == ARG, (name, x)
        for y in outs[name]:
            assert call(name, saved=apart[y]) == ARG, (name, y)
        if not torch.cuda.is_available():
            assert call(name) not in (rh.RL_OK, ARG), name        # (no device)
            for y in ("loss", "mass"):
                assert call(name, **{y: apart["dloss"]}) not in (rh.RL_OK, ARG), (name, y)
            for y in outs[name]:
                assert call(name, **{y: apart["ids"] + 40}) not in (rh.RL_OK, ARG), (name, y)
    for y in ("loss", "mass"):
        assert call("fwd_bwd", **{y: apart["dlogits"] + 15996}) == ARG
    assert call("fwd", loss=apart["mass"] + 12) == ARG
    if not torch.cuda.is_available():
        assert call("bwd", loss=apart["ids"], mass=apart["logits"]) not in (rh.RL_OK, ARG)      # (not of the backward)
