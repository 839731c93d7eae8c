"""Page plans at the borders of what their arguments may be (whole numbers: every value equal)."""
import numpy as np
import pytest
import torch

import lm_head_gb300 as rh
from test_gpu_pages import LENGTHS, make, run_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,G", [(5, 3), (3000, 1500)])
def test_group_offsets_that_do_not_add_up_set_status(R, G):
    q, ctx, table, pool, used, page, n_pages, T, go, pl = make(R, 3, 40, 16, R, G)
    p, _ = run_plan(q, ctx, table, pool, used, page, n_pages, T, go, pl)
    assert p.status_bits() == 0
    for i, bad in ((G, R + 1), (0, -1), (G - 1, R + 7)):
        b = np.array(go)
        b[i] = bad
        p, _ = run_plan(q, ctx, table, pool, used, page, n_pages, T, b, pl)
        assert p.status_bits() == LENGTHS, rh.status_names(p.status_bits())


@pytest.mark.parametrize("R,q_max,G", [(3, 1, 2), (5000, 4, 40), (9, 5000, 4)])
def test_lengths_in_place(R, q_max, G):
    """kv_lens in the place of ctx_lens: what separate lengths give, also where several blocks would
    share the step."""
    q, ctx, table, pool, used, page, n_pages, T, go, pl = make(R, q_max, 40, 16, R, G)
    c = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    args = dict(page_size=page, n_pages=n_pages, n_tokens=T, free_used=c([used]), group_offsets=c(go), prefix_lens=c(pl))
    t0, t1, lens = c(table), c(table), c(ctx)
    a = rh.rl_page_plan(c(q), c(ctx), t0, c(pool), **args)
    e = lambda n, dt: torch.empty(n, dtype=dt, device="cuda")  # noqa: E731
    b = rh.rl_page_plan(c(q), lens, t1, c(pool), out=rh.PagePlan(
        e(R + 1, torch.int32), lens, e(T, torch.int64), e(T, torch.int32), e(1, torch.int32),
        torch.zeros(1, dtype=torch.int32, device="cuda")), **args)
    assert a.status_bits() == b.status_bits() == 0 and torch.equal(t0, t1)
    for x, y in ((a.cu_q, b.cu_q), (a.kv_lens, lens), (a.slot_map, b.slot_map), (a.positions, b.positions), (a.free_used, b.free_used)):
        assert torch.equal(x, y)
