"""A wait that runs out in the middle of a block's run of items: what the run holds from
there on is NaN or right, never something else, and the workspace and the GPU stay usable."""
import ctypes
import os
import subprocess
import time

import pytest
import torch
from test_gpu_attn import Attn, Q  # noqa: F401
from test_gpu_lost_copies import CSRC, HERE, vp
from test_gpu_lost_tiles import build

pytestmark = pytest.mark.gpu


def run(lib, a, limit=40):
    a.out.fill_(7.0)
    a.lse.fill_(7.0)
    torch.cuda.synchronize()
    begin = time.monotonic()
    assert lib.attend(ctypes.byref(a.cfg), ctypes.byref(a.seqs), a.m, *vp(a.q, a.k, a.v, a.out, a.lse, a.ws)) == 0
    torch.cuda.synchronize()
    assert time.monotonic() - begin < limit


def nan_or(a, want):
    """where lse is NaN; all else is as wanted"""
    bad = torch.isnan(a.lse)
    each = bad[:, :, None].expand(-1, -1, a.dim).reshape(a.m, -1)
    assert torch.equal(a.lse[~bad], want[1][~bad]) and torch.equal(a.out[~each], want[0][~each])
    assert torch.isnan(a.out[each]).all() and not bad.all()
    return bad


@pytest.mark.parametrize("c", [
    dict(new=[1] * 1600, kv=[1 + i % 32 for i in range(1600)], heads=4, kv_heads=2, dim=128, page=32),
    dict(new=[1] * 900, kv=[33 + i % 30 for i in range(900)], heads=6, kv_heads=2, dim=64, page=64, t="f16"),
], ids=["one-tile", "two-tiles"])
def test_short_items_after_a_lost_copy(Q, tmp_path_factory, c):  # noqa: F811
    """each block has ten and more items of fewer tiles than its ring holds, so that a copying warp has much
    left to do when a wait runs out, and some computing warps have waited for nothing yet"""
    lib = build(tmp_path_factory.getbasetemp(), "k_attn_rows", False)
    a = Attn(Q, seed=5, **c)
    run(lib, a)
    a.check(only=range(0, a.batch, 97))
    want = a.out.clone(), a.lse.clone()
    for hit in (0, a.batch // 2 + 3, a.batch - 30):
        assert lib.lose(int(a.table[hit, 0])) == 0
        run(lib, a)
        assert nan_or(a, want)[hit].all()
        assert Q.moe_v41_read_status(a.ws, clear=True) == Q.MOE_STATUS_TIMEOUT
        assert lib.lose(-1) == 0
        run(lib, a)
        assert torch.equal(a.out, want[0]) and torch.equal(a.lse, want[1])
        assert Q.moe_v41_read_status(a.ws) == 0


def build_items(tmp):
    import quantized_mixture_experts_router_gb300.build as qb
    so = os.path.join(str(tmp), "lost_items.so")
    if not os.path.exists(so):
        subprocess.run([qb.NVCC, *qb.ARCH, *qb.FLAGS, "-I", CSRC, "-DKERNEL=\"k_attn_tiles.cu\"", "-DTILES", "-shared",
                        os.path.join(HERE, "lost_items.cu"), "-o", so, "-lcudart"], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("c", [
    dict(new=[40] * 600, kv=[60 + i % 90 for i in range(600)], heads=4, kv_heads=2, dim=128, page=16),
    dict(new=[300, 20, 600], kv=[30000, 500, 14000], heads=4, kv_heads=2, dim=64, page=64, t="f16"),
], ids=["many-items", "cut-items"])
def test_items_that_are_never_told(Q, tmp_path_factory, c):  # noqa: F811
    """the warps that wait for them agree on the last one that was told, the rest of the run is NaN, and parts of
    items that other blocks join are counted all the same"""
    lib = build_items(tmp_path_factory.getbasetemp())
    a = Attn(Q, seed=6, **c)
    run(lib, a)
    a.check(only=range(0, a.batch, 97))
    want = a.out.clone(), a.lse.clone()
    # many: eight items a block, and the run's end.  cut: the run of block 0 is a part of one item, so that its end is
    # lost; those of the others are the end of an item and the beginning of the next, or two whole ones
    ends = [(0, 1), (138, 2)] if a.batch < 100 else [(100, 8)]           # nothing but the run's end gets lost
    many = [(0, 1), (70, 5), (151, 2), (33, -1), (100, 8)]
    cut = [(0, 1), (28, 1), (56, 1), (85, 1), (138, 1), (138, 2)]
    for block, item in many if a.batch > 100 else cut:
        assert lib.lose_item(block, item) == 0
        run(lib, a)
        assert nan_or(a, want).any() != ((block, item) in ends)
        assert Q.moe_v41_read_status(a.ws, clear=True) == Q.MOE_STATUS_TIMEOUT
        assert lib.lose_item(-1, 0) == 0
        run(lib, a)
        assert torch.equal(a.out, want[0]) and torch.equal(a.lse, want[1])
        assert Q.moe_v41_read_status(a.ws) == 0
