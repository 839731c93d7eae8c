"""rl_prefix_attn where its kernels differ from one another or meet what they may not follow.

The bars are those of test_gpu_prefix_attn.py.
"""
import pytest
import torch

import lm_head_gb300 as rh  # noqa: F401
from test_gpu_prefix_attn import BF, HF, Case

pytestmark = pytest.mark.gpu

# a step whose rows are done by tiles of 16, by one tile of up to 128 rows, and by two such tiles
KINDS = [("warp", dict(groups=[3], prefixes=[70], q_lens=[1] * 3, kv_lens=[1, 17, 64])),
         ("warp, one part", dict(groups=[], prefixes=[], q_lens=[1, 3], kv_lens=[200, 40])),
         ("keys", dict(groups=[17], prefixes=[300], q_lens=[1] * 17, kv_lens=[1 + 9 * i for i in range(17)])),
         ("keys, one part", dict(groups=[], prefixes=[], q_lens=[20, 11], kv_lens=[150, 11])),
         ("rows", dict(groups=[2], prefixes=[131], q_lens=[130, 70], kv_lens=[130, 400])),
         ("rows, one part", dict(groups=[], prefixes=[], q_lens=[140], kv_lens=[190]))]


def make(kind, D=64, page=16, dtype=BF, seed=1):
    return Case(Hq=8, Hkv=2, D=D, page=page, dtype=dtype, seed=seed, **dict(KINDS)[kind])


@pytest.mark.parametrize("kind", [k for k, _ in KINDS])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF)])
def test_scale_zero_is_the_mean_of_the_values(kind, D, dtype):
    c = make(kind, D, dtype=dtype)
    c.scale = 0.0
    c.check()
