"""A copy of the cache that never lands: the attention kernels' bounded waits run out,
what depended on it is NaN, the rest is right, the status says so, and the workspace
and the GPU stay usable.  The kernels are built here with a copy that the test drops
(lost_tiles.cu)."""
import ctypes
import os
import subprocess
import time

import pytest
import torch
from test_gpu_attn import Attn, Q, desc  # noqa: F401
from test_gpu_lost_copies import CSRC, HERE, vp

pytestmark = pytest.mark.gpu


def build(tmp, kernel, tiles):
    import quantized_mixture_experts_router_gb300.build as qb
    so = os.path.join(str(tmp), f"lost_{kernel}.so")
    if not os.path.exists(so):
        subprocess.run([qb.NVCC, *qb.ARCH, *qb.FLAGS, "-I", CSRC, f"-DKERNEL=\"{kernel}.cu\"", *(["-DTILES"] if tiles else []),
                        "-shared", os.path.join(HERE, "lost_tiles.cu"), "-o", so, "-lcudart"], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("kernel,c", [
    ("k_attn_rows", dict(new=[1] * 40, kv=[300 + 11 * i for i in range(40)], heads=8, kv_heads=2, dim=128, page=16)),
    ("k_attn_rows", dict(new=[1, 2, 1], kv=[20000, 50, 300], heads=8, kv_heads=1, dim=64, page=32, t="f16")),
    ("k_attn_tiles", dict(new=[300, 20, 600], kv=[2000, 500, 600], heads=4, kv_heads=2, dim=128, page=16)),
    ("k_attn_tiles", dict(new=[30, 1, 400], kv=[9000, 50, 3000], heads=6, kv_heads=2, dim=64, page=64, t="f16")),
], ids=str)
def test_a_lost_copy_of_the_cache(Q, tmp_path_factory, kernel, c):  # noqa: F811
    lib = build(tmp_path_factory.getbasetemp(), kernel, kernel.endswith("tiles"))
    a = Attn(Q, seed=2, **c)

    def call():
        a.out.fill_(7.0)
        a.lse.fill_(7.0)
        torch.cuda.synchronize()
        begin = time.monotonic()
        assert lib.attend(ctypes.byref(a.cfg), ctypes.byref(a.seqs), a.m, *vp(a.q, a.k, a.v, a.out, a.lse, a.ws)) == 0
        torch.cuda.synchronize()
        assert time.monotonic() - begin < 40

    call()
    a.check()
    want = a.out.clone(), a.lse.clone()
    hit = len(a.new) - 1
    rows = slice(a.cu[hit], a.cu[hit + 1])
    for at in (0, -(-a.kv[hit] // a.page) - 1):                        # the sequence's first page, and its last
        assert lib.lose(int(a.table[hit, at])) == 0
        call()
        bad = torch.isnan(a.lse)
        last = rows.stop - 1                                             # a row that sees either page
        assert bad[last].all() and torch.isnan(a.out[last]).all()
        good = ~bad[:, :, None].expand(-1, -1, a.dim).reshape(a.m, -1)
        assert good.any() and torch.equal(a.out[good], want[0][good]) and torch.isnan(a.out[~good]).all()
        assert torch.equal(a.lse[~bad], want[1][~bad])
        assert Q.moe_v41_read_status(a.ws, clear=True) == Q.MOE_STATUS_TIMEOUT
        assert lib.lose(-1) == 0                                         # the same kernel with every copy
        call()
        assert torch.equal(a.out, want[0]) and torch.equal(a.lse, want[1])
        assert Q.moe_v41_read_status(a.ws) == 0
