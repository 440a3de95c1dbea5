"""The operators around the MoE layer on the GPU where their work is walked
through in parts: several tiles a block, ranges and places at the ends of what
the calls take.  Tolerances as in test_gpu_ops.py."""
import pytest
import torch
from test_gpu_ops import Q, Q4  # noqa: F401

pytestmark = pytest.mark.gpu


# 313 row tiles of 128 and one or two token tiles, more than there are SMs: blocks walk through several tiles.  Token
# tiles end below and above 128; rows end inside a stage, a group, and after odd numbers of groups.
@pytest.mark.parametrize("m", [100, 130, 300, 390, 512])
@pytest.mark.parametrize("k,group", [(352, 128), (160, 64), (96, 64), (352, 32), (160, 32), (1056, 128)])
def test_q4_many_tiles_a_block(Q, m, k, group):  # noqa: F811
    t = Q4(Q, m, 40001, k, group, zeros=True, x="bf16" if m % 4 else "f16", pado=3, seed=m + k + group)
    t.call()
    t.check()
    first = t.out.clone()
    for _ in range(3):
        t.out.zero_()
        t.call()
        assert torch.equal(t.out, first)
