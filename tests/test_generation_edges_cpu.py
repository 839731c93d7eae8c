"""Generation operators, host side: arguments refused before any device work (no GPU needed)."""
import lm_head_gb300 as rh
from lm_head_gb300 import generation as gen
from test_generation_cpu import FAKE, _fill, _refused, lib  # noqa: F401


def test_page_plan_refuses_lengths_that_share_memory_with_its_outputs(lib):  # noqa: F811
    names = ("q_lens", "ctx_lens", "block_table", "free_pages", "free_used", "free_used_out", "group_offsets", "prefix_lens",
             "cu_q", "kv_lens", "slot_map", "positions")
    apart = {n: FAKE * (i + 1) for i, n in enumerate(names)}

    def make(**kw):
        return _fill(gen.RlPagePlanArgs, **{**dict(R=4, T=8, table_width=2, n_free=8, G=2, n_pages=8, page_size=16), **apart, **kw})
    arg = rh.RL_ERR_ARG
    _refused(lib, "rl_page_plan", make, [
        (dict(kv_lens=apart["q_lens"]), arg), (dict(kv_lens=apart["ctx_lens"] + 4), arg),
        (dict(kv_lens=apart["ctx_lens"] - 12), arg), (dict(cu_q=apart["ctx_lens"]), arg), (dict(cu_q=apart["q_lens"] - 16), arg)])
