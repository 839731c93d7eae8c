"""Verification of drafts, host side: what is refused before any device work, and the definition's own arithmetic."""
import ctypes

import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from lm_head_gb300 import verify as vf
from test_generation_cpu import FAKE, _fill, _refused, lib  # noqa: F401
from verify_ref import Side, verify_reference

ARG, UNS = rh.RL_ERR_ARG, rh.RL_ERR_UNSUPPORTED


def make(**kw):
    far = FAKE + (1 << 20)
    return _fill(vf.RlVerifyArgs, **{**dict(R=4, T=8, V=1000, target_n_rows=8, target_row_stride=1000, target_nnz=10, draft_n_rows=8,
                                            draft_row_stride=1000, draft_nnz=10, target_dtype=0, draft_dtype=1, tokens=far,
                                            keep_lens=far, ctx_lens=FAKE), **kw})


def test_refusals(lib):  # noqa: F811
    both = [(k, v, w) for k, v, w in (("n_rows", -1, ARG), ("nnz", -1, ARG), ("n_rows", 1 << 31, UNS), ("row_stride", 999, ARG),
                                      ("ids", None, ARG), ("logq", None, ARG), ("replayed", None, ARG), ("logits", FAKE + 1, ARG))]
    changes = [({s + k: v}, w) for s in ("target_", "draft_") for k, v, w in both]
    changes += [(dict(R=-1), ARG), (dict(T=-1), ARG), (dict(V=0), ARG), (dict(V=(1 << 20) + 1), UNS), (dict(R=1 << 28), UNS),
                (dict(T=1 << 31), UNS), (dict(target_dtype=3), UNS), (dict(draft_dtype=-1), UNS),
                (dict(target_logits=None, target_offsets=None), ARG), (dict(cu_q=None), ARG), (dict(step_tokens=None), ARG),
                (dict(u=None), ARG), (dict(u_next=None), ARG), (dict(tokens=None), ARG), (dict(accepted=None), ARG),
                (dict(tokens=FAKE + 4), ARG), (dict(keep_lens=FAKE + 4), ARG)]
    _refused(lib, "rl_verify", make, changes, tail=(FAKE, 1 << 40))
    a = make(T=100000, target_n_rows=100000, draft_n_rows=100000)
    assert lib.rl_verify(ctypes.byref(a), FAKE, 64, FAKE, None) == rh.RL_ERR_WORKSPACE
    assert lib.rl_verify(ctypes.byref(a), None, 1 << 40, FAKE, None) == ARG
    assert lib.rl_verify(ctypes.byref(a), FAKE + 8, 1 << 40, FAKE, None) == ARG
    bad = make(V=0)
    assert lib.rl_verify_workspace_bytes(ctypes.byref(bad)) == 0 and lib.rl_verify_workspace_bytes(None) == 0
    assert ctypes.sizeof(vf.RlVerifyArgs) == (7 + 20 + 1 + 5) * 8


def test_outputs_that_share_memory_with_inputs(lib):  # noqa: F811
    apart = {n: FAKE + (k << 16) for k, n in enumerate(("cu_q", "step_tokens", "u", "u_next", "ctx_lens", "tokens", "logq", "accepted",
                                                        "keep_lens"))}

    def call(**kw):
        a = make(**{**apart, **kw})
        return lib.rl_verify(ctypes.byref(a), FAKE, 1 << 40, FAKE, None)
    if not torch.cuda.is_available():
        assert call() not in (rh.RL_OK, ARG) and call(keep_lens=apart["ctx_lens"]) != ARG      # (no device)
    for x in ("cu_q", "step_tokens", "u", "u_next"):
        for y in ("tokens", "logq", "accepted", "keep_lens"):
            assert call(**{y: apart[x] + 4}) == ARG, (x, y)
    assert call(accepted=apart["ctx_lens"]) == ARG


def test_binding_refuses_host_tensors_and_missing_rows():
    i, f = torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    with pytest.raises(rh.RLHeadError):
        rh.rl_verify(i, i[:2], f, f[:1], rh.Dist(logits=torch.zeros(3, 10)), vocab=10)
    with pytest.raises(rh.RLHeadError):
        rh.rl_verify(i, i[:2], f, f[:1], rh.Dist(), vocab=10)
    with pytest.raises(rh.RLHeadError):
        rh.rl_verify(i, i[:2], f, f[:1], None, vocab=10)


def test_the_rule_gives_the_targets_distribution():
    """Accept-or-redraw over a fine grid of random numbers: the first token's distribution is p, by arithmetic."""
    V, n = 4, 64
    z, zd = np.array([[0.3, -1.0, 0.9, 0.0]]), np.array([[1.0, 0.2, -0.5, 0.1]])
    p, q = (np.exp(x[0]) / np.exp(x[0]).sum() for x in (z, zd))
    got = np.zeros(V)
    rows = np.zeros(2, int)
    for x in range(V):
        for i in range(n):
            for k in range(n):
                t = verify_reference([0, x], [0, 2], [(i + 0.5) / n, 0], [(k + 0.5) / n], Side(V, z, rows=rows), Side(V, zd, rows=rows))
                got[t["tokens"][0]] += q[x] / n / n
    assert np.abs(got - p).max() < 2.0 / n          # the grid's own coarseness


def test_outputs_that_share_memory_with_the_distributions(lib):  # noqa: F811
    """Each array of either side, its first and its last element; outputs between the rows of the logits are sound."""
    names = ["cu_q", "step_tokens", "u", "u_next", "ctx_lens", "tokens", "logq", "accepted", "keep_lens"]
    size = dict(logits=8 * 1000 * 4, temperature=32, offsets=72, ids=40, logq=40, replayed=8, rows=32)
    names += [s + n for s in ("target_", "draft_") for n in size]
    apart = {n: FAKE + (k << 16) for k, n in enumerate(names)}

    def call(**kw):
        a = make(**{**apart, **kw})
        return lib.rl_verify(ctypes.byref(a), FAKE + (1 << 28), 1 << 40, FAKE + (1 << 27), None)
    outs = ("tokens", "logq", "accepted", "keep_lens")
    for s in ("target_", "draft_"):
        for n, z in size.items():
            last = 8 * 1000 * 2 if (s, n) == ("draft_", "logits") else z
            for y in outs:
                assert call(**{y: apart[s + n]}) == call(**{y: apart[s + n] + last // 4 * 4 - 4}) == ARG, (s, n, y)
    for y in ("tokens", "logq", "accepted"):
        assert call(**{y: apart["ctx_lens"] + 12}) == ARG, y
    if not torch.cuda.is_available():
        assert call() not in (rh.RL_OK, ARG) and call(keep_lens=apart["ctx_lens"]) not in (rh.RL_OK, ARG)     # (no device)
        for n, z in size.items():       # just past each
            assert call(tokens=apart["target_" + n] + (z + 3) // 4 * 4) not in (rh.RL_OK, ARG), n
        assert call(target_row_stride=1100, tokens=apart["target_logits"] + 4 * 1040) not in (rh.RL_OK, ARG)
        assert call(draft_logits=None, draft_offsets=None, tokens=apart["draft_ids"]) not in (rh.RL_OK, ARG)
    assert call(target_row_stride=1100, tokens=apart["target_logits"] + 4 * 1098) == ARG
