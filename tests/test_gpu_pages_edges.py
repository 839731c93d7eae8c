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
