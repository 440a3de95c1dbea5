"""A copy that never lands: the kernel's bounded wait runs out, the rows that
depended on it are marked, the others are right, and the GPU stays usable.
The kernels are built here with a copy that the test drops (lost_copies.cu)."""
import ctypes
import os
import subprocess
import time

import pytest
import torch
from test_gpu_ops import Lp, Norm, Q, Q4  # noqa: F401

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "quantized_mixture_experts_router_gb300", "csrc")


def build(tmp, kernel, define):
    import quantized_mixture_experts_router_gb300.build as qb
    so = os.path.join(str(tmp), define.lower() + ".so")
    if not os.path.exists(so):
        subprocess.run([qb.NVCC, *qb.ARCH, *qb.FLAGS, "-I", CSRC, f"-DKERNEL=\"{kernel}\"", f"-D{define}", "-shared",
                        os.path.join(HERE, "lost_copies.cu"), "-o", so, "-lcudart"], check=True)
    lib = ctypes.CDLL(so)
    lib.lose.argtypes = [ctypes.c_uint64]
    return lib


def vp(*tensors):
    return [ctypes.c_void_p(t.data_ptr()) for t in tensors]


def spaced(rows, first, m):
    """rows are first, first + step, ... up to m"""
    step = rows[1] - rows[0] if len(rows) > 1 else m
    return rows == list(range(first, m, step)) and step > 1


@pytest.mark.parametrize("lose", ["y", "h"])
def test_norm_marks_the_rows_of_a_lost_copy(Q, tmp_path_factory, lose):  # noqa: F811
    lib = build(tmp_path_factory.getbasetemp(), "k_norm.cu", "NORM")
    m, dim, at = 900, 5120, 200
    t = Norm(Q, m, dim, y="f32", h="f32", seed=1)
    t.post_w = t.pre_w = None
    t.call(post_w=None, pre_w=None)
    want = t.h_out.clone(), t.x_out.clone()
    t.h_out.fill_(7.0)
    t.x_out.fill_(7.0)
    torch.cuda.synchronize()
    assert lib.lose(getattr(t, lose)[at].data_ptr()) == 0
    begin = time.monotonic()
    assert lib.block_norm(ctypes.byref(t.cfg), m, *vp(t.y, t.h, t.h_out, t.x_out)) == 0
    torch.cuda.synchronize()
    assert time.monotonic() - begin < 20
    bad = torch.isnan(t.h_out).any(1)
    assert spaced(bad.nonzero()[:, 0].tolist(), at, m)
    assert torch.isnan(t.h_out[bad]).all() and torch.isnan(t.x_out[bad]).all()
    assert torch.equal(t.h_out[~bad], want[0][~bad]) and torch.equal(t.x_out[~bad], want[1][~bad])
    assert lib.lose(0) == 0                                     # the same kernel with every copy
    assert lib.block_norm(ctypes.byref(t.cfg), m, *vp(t.y, t.h, t.h_out, t.x_out)) == 0
    torch.cuda.synchronize()
    assert torch.equal(t.h_out, want[0]) and torch.equal(t.x_out, want[1])


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_logprob_marks_the_rows_of_a_lost_copy(Q, tmp_path_factory, t):  # noqa: F811
    """the first piece of one row of a block that walks through several, and of a row that a cluster shares"""
    lib = build(tmp_path_factory.getbasetemp(), "k_logprob.cu", "LOGPROB")
    for m, v, at in ((2000, 6400, 900), (3, 64000, 1)):
        c = Lp(Q, m, v, t, 5, seed=3)
        c.call()
        floats, ints = (c.logprob, c.lse, c.entropy, c.top), (c.rank, c.ids)
        want = [o.clone() for o in floats + ints]
        for o in floats + ints:
            o.fill_(7)
        torch.cuda.synchronize()

        def call():
            begin = time.monotonic()
            assert lib.token_logprobs(ctypes.byref(c.cfg), *vp(c.x), m,
                                      *vp(c.target, c.logprob, c.rank, c.lse, c.entropy, c.top, c.ids)) == 0
            torch.cuda.synchronize()
            assert time.monotonic() - begin < 20

        assert lib.lose(c.x[at].data_ptr()) == 0
        call()
        bad = torch.isnan(c.lse)
        assert spaced(bad.nonzero()[:, 0].tolist(), at, m)
        for o, w in zip(floats + ints, want):
            assert torch.equal(o[~bad], w[~bad])
            assert torch.isnan(o[bad]).all() if o.is_floating_point() else (o[bad] == -1).all()
        assert lib.lose(0) == 0                                    # the same kernel with every copy
        call()
        assert all(torch.equal(o, w) for o, w in zip(floats + ints, want))


# row tiles shared by many blocks; whole row tiles a block, two tokens; runs of several boxes
@pytest.mark.parametrize("m,n,k,group,block", [(1, 64, 32768, 128, 3), (2, 20001, 512, 64, 7), (8, 700, 5120, 32, 9)])
def test_q4_marks_the_rows_of_a_lost_copy(Q, tmp_path_factory, m, n, k, group, block):  # noqa: F811
    """the outputs of the row tiles that the block's first warp has a part of are NaN; the workspace stays ready"""
    lib = build(tmp_path_factory.getbasetemp(), "k_q4.cu", "LINEAR")
    t = Q4(Q, m, n, k, group, seed=5)
    t.call()
    want = t.out.clone()

    def call():
        t.out.fill_(7.0)
        torch.cuda.synchronize()
        begin = time.monotonic()
        assert lib.q4_linear(ctypes.byref(t.cfg), *vp(t.x), m, *vp(t.w, t.scales, t.out, t.ws)) == 0
        torch.cuda.synchronize()
        assert time.monotonic() - begin < 20

    for _ in range(2):
        assert lib.lose(block + 1) == 0
        call()
        bad = torch.isnan(t.out).any(0)
        tiles = (bad.nonzero()[:, 0] // 32).unique().tolist()
        assert 1 <= len(tiles) <= 3 and tiles == list(range(tiles[0], tiles[-1] + 1))
        rows = torch.arange(n, device="cuda") // 32
        assert torch.equal(bad, (rows >= tiles[0]) & (rows <= tiles[-1])) and torch.isnan(t.out[:, bad]).all()
        assert torch.equal(t.out[:, ~bad], want[:, ~bad])
        assert Q.moe_v41_read_status(t.ws, clear=True) == Q.MOE_STATUS_TIMEOUT
        assert lib.lose(0) == 0
        call()
        assert torch.equal(t.out, want)
        assert Q.moe_v41_read_status(t.ws) == 0
