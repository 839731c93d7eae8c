"""Distillation at the ends of the range: finite masks, small temperatures, probabilities that underflow."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from test_gpu_distill import DT, KINDS, NONFINITE, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,tail", KINDS)
@pytest.mark.parametrize("dtype,V", [("fp32", 5003), ("bf16", 5003), ("fp32", 151936), ("bf16", 151936)])
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e20, None])
def test_rows_masked_by_a_finite_number(kind, tail, dtype, V, mask):
    """All but a few tokens masked, whole slices of a row among them, with and without a token of the rest that is not."""
    N = 6
    mask = torch.finfo(DT[dtype]).min if mask is None else mask
    for T in (1.0, 0.3):
        c = make(N, V, dtype, np.array([5, 9, 3, 70, 8, 2]), T, tail, seed=3)
        off, ids = c["off"].tolist(), c["ids"].long()
        for r in range(N):
            keep = torch.zeros(V, dtype=torch.bool, device="cuda")
            keep[ids[off[r]:off[r + 1]]] = True
            if r % 3:
                keep[[11, V // 2]] = True
            if r == 4:
                keep[:V // 3] = True
            c["z"][r][~keep] = mask
        check(c, rh.DistillParams(kind=kind, tail=tail, temperature=T, beta=0.4), dtype)


@pytest.mark.parametrize("kind,tail", KINDS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale,T", [(1e4, 2.0 ** -20), (30.0, 2.0 ** -20), (1e10, 1.0), (3e6, 0.25)])
def test_exponents_of_any_size(kind, tail, dtype, scale, T):
    """Logits over the temperature from 2^24 to 2^34, the largest in the support and outside it, alone and several times."""
    N, V = 8, 3001
    c = make(N, V, dtype, np.array([5, 9, 3, 70, 8, 2, 4, 6]), 1.0, tail, seed=5, scale=1.0)
    off, ids = c["off"].tolist(), c["ids"].long()
    c["z"].mul_(scale)
    for r in range(N):
        top = c["z"][r].float().max() * 1.25
        S = ids[off[r]:off[r + 1]]
        other = [j for j in (100, 2000, 2999, 17, 18) if j not in S.tolist()]
        if r % 4 < 2:
            c["z"][r, S[0]] = top.to(DT[dtype])
        if r % 4 == 1:
            c["z"][r, S[1]] = top.to(DT[dtype])
        if r % 4:
            c["z"][r, other[:r % 4]] = top.to(DT[dtype])
    check(c, rh.DistillParams(kind=kind, tail=tail, temperature=T, beta=0.4), dtype)


@pytest.mark.parametrize("kind,tail", KINDS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("beta", [0.4, 0.999])
def test_tokens_that_neither_side_gives(kind, tail, dtype, beta):
    """Entries of the support whose probabilities underflow on both sides, on one of them, and rows of little else."""
    N, V = 6, 2000
    c = make(N, V, dtype, np.array([6, 6, 6, 6, 300, 6]), 1.0, tail, seed=8)
    off, ids = c["off"].tolist(), c["ids"].long()
    for r in range(N):
        S = ids[off[r]:off[r + 1]]
        q = c["q"][off[r]:off[r + 1]]
        if r == 4:
            # (above the 64-bit reference's own underflow)
            q[10:] = torch.linspace(-110, -650, len(S) - 10).cuda()
            c["z"][r, S[10:]] = torch.linspace(-650, -130, len(S) - 10).cuda().to(DT[dtype])
            continue
        c["z"][r, S[1]] = -130.0
        q[1] = (-120.0, -1e4, -106.0, -3e4, 0, -104.5)[r]
        c["z"][r, S[2]] = -1e4
        q[3] = -150.0
    check(c, rh.DistillParams(kind=kind, tail=tail, beta=beta), dtype)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_probabilities_next_to_the_least_float(kind, dtype):
    """Entries whose student's probability is subnormal while their weight relative to the row's largest is not, beside a teacher's
    probability of the same size and of none."""
    N, V = 8, 3000
    c = make(N, V, dtype, np.full(N, 40), 1.0, True, seed=9, scale=0.1)
    off, ids = c["off"].tolist(), c["ids"].long()
    for r in range(N):
        S = ids[off[r]:off[r + 1]]
        c["z"][r, S[5:35]] = torch.linspace(-86.5, -78, 30).cuda().to(DT[dtype])
        c["q"][off[r] + 5:off[r] + 35] = torch.linspace(-80, -95, 30).cuda() if r % 2 else -200.0
    check(c, rh.DistillParams(kind=kind, tail=True, beta=0.3), dtype)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("dtype,V", [("fp32", 1000), ("bf16", 1000), ("fp16", 1000), ("fp32", 70001), ("bf16", 151936)])
@pytest.mark.parametrize("T", [1.0, 0.1])
def test_a_rest_far_below_the_support(kind, dtype, V, T):
    """Gaps of up to 700 temperatures between the support's logits and the rest's, and the other way round: where the student gives
    the rest next to nothing, the forward kind's teacher still wants its share of it."""
    gaps = [20, 55, 60, 80, 86, 88, 90, 95, 100, 104, 110, 200, 700, -60, -90, -200]
    N = len(gaps)
    c = make(N, V, dtype, np.full(N, 7), T, True, seed=6, scale=T)
    off, ids = c["off"].tolist(), c["ids"].long()
    c["dl"][:] = 0.7
    for r, g in enumerate(gaps):
        S = ids[off[r]:off[r + 1]]
        c["z"][r, S] = (c["z"][r, S].float() * 0.2 + g * T).to(DT[dtype])
        if r % 2:           # (a teacher who gives the rest some tenths, and one who gives it a hundredth)
            c["q"][off[r]:off[r + 1]] = torch.log(torch.tensor([0.1, 0.2, 0.05, 0.1, 0.04, 0.01, 0.1])).cuda()
        else:
            c["q"][off[r]:off[r + 1]] = torch.log(torch.tensor([0.3, 0.4, 0.05, 0.1, 0.04, 0.05, 0.05])).cuda()
    o, d = check(c, rh.DistillParams(kind=kind, tail=True, temperature=T, beta=0.4), dtype)
    if kind == "forward":   # (the rest's gradient sums to P_0 - t_0)
        rest = d.float()
        for r in range(13):
            rest[r, ids[off[r]:off[r + 1]]] = 0
        share = torch.tensor([0.01, 0.4]).repeat(N)[:13].cuda() * 0.7 / T
        assert (((rest[:13].double().sum(1) + share) / share).abs() <= (0.02 if dtype != "fp16" else 0.3)).all()


@pytest.mark.parametrize("kind,tail", KINDS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [0.7, 2.0 ** -20])
def test_support_tokens_masked_by_the_lowest_number(kind, tail, dtype, T):
    """The quotient of the type's lowest number and T is no float: the token has no probability, as one of -inf."""
    N, V = 5, 1500
    c = make(N, V, dtype, np.full(N, 8), 1.0, tail, seed=7)       # (every token of it wanted)
    off, ids = c["off"].tolist(), c["ids"].long()
    low = c["z"].clone()
    for r in range(N):
        c["z"][r, ids[off[r] + r]] = torch.finfo(DT[dtype]).min
        low[r, ids[off[r] + r]] = float("-inf")
    p = rh.DistillParams(kind=kind, tail=tail, temperature=T, beta=0.4)
    if kind != "forward":       # (there the loss is of that size, or inf)
        check(c, p, dtype)
    args = (c["off"], c["ids"], c["q"], c["dl"], p)
    o, d = rh.rl_distill_fwd_bwd(c["z"], *args)
    want, wd = rh.rl_distill_fwd_bwd(low, *args)
    assert torch.equal(o.loss, want.loss) and torch.equal(o.mass, want.mass) and torch.equal(d, wd)
    assert o.status_bits() == want.status_bits() == (NONFINITE if kind == "forward" else 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [1001, 70001])
def test_gradients_beside_the_logits_in_one_buffer(dtype, V):
    c = make(5, V, dtype, np.array([3, 0, 5, 20, 1]), 1.0, True, seed=2)
    args = (c["off"], c["ids"], c["q"])
    p = rh.DistillParams(kind="reverse", tail=True)
    for first in (0, V):
        buf = torch.zeros(5, 2 * V, dtype=DT[dtype], device="cuda")
        z, g = buf[:, first:first + V], buf[:, V - first:2 * V - first]
        z.copy_(c["z"])
        want, wd = rh.rl_distill_fwd_bwd(z, *args, c["dl"], p)
        o, d = rh.rl_distill_fwd_bwd(z, *args, c["dl"], p, dlogits=g)
        assert d is g and torch.equal(o.loss, want.loss) and torch.equal(g, wd) and torch.equal(z, c["z"])
        f = rh.rl_distill_fwd(z, *args, p)
        want2, _ = rh.rl_distill_bwd(z, *args, p, f.saved, c["dl"])
        g.zero_()
        rh.rl_distill_bwd(z, *args, p, f.saved, c["dl"], dlogits=g)
        assert torch.equal(g, want2) and torch.equal(z, c["z"])


def test_the_loss_in_dloss_s_place():
    c = make(300, 4099, "bf16", np.arange(300) % 40, 1.0, True)
    args = (c["z"], c["off"], c["ids"], c["q"])
    p = rh.DistillParams(kind="jsd", tail=True)
    want, wd = rh.rl_distill_fwd_bwd(*args, c["dl"], p)
    o, _ = rh.rl_distill_fwd_bwd(*args, c["dl"], p)
    o.loss = c["dl"].clone()
    o, d = rh.rl_distill_fwd_bwd(*args, o.loss, p, out=o)
    assert torch.equal(o.loss, want.loss) and torch.equal(d, wd) and torch.equal(o.mass, want.mass)
