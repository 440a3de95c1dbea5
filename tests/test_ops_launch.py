"""The operators' launchers without a GPU: the library's objects linked with a
runtime that launches nothing (fake_cudart.cc)."""
import ctypes
import os
import subprocess

import pytest
from test_ops_args import Q  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture
def fake(Q, tmp_path):  # noqa: F811
    """a library of its own for every test: what the launchers remember starts empty"""
    lib_dir = os.path.dirname(Q.SO)
    objs = [os.path.join(lib_dir, f"{o}.o") for o in ("k_logprob", "k_norm", "k_q4", "k_q4_gemm", "ops_capi")]
    so = str(tmp_path / "fake.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", "/usr/local/cuda/include", "-Wl,-Bsymbolic",
                    os.path.join(HERE, "fake_cudart.cc"), *objs, "-o", so, "-lpthread"], check=True)
    return ctypes.CDLL(so)


def counts(lib):
    out = (ctypes.c_int * 3)()
    lib.counts(out)
    return list(out)


def test_calls_from_many_threads_on_two_devices(fake):
    fake.set_registers(96)
    threads, calls = 8, 2000
    assert fake.call_from_threads(threads, calls) == 0
    launches, bad, _ = counts(fake)
    assert launches == threads * calls * 4 and bad == 0


def test_q4_many_tokens_whatever_registers_the_compiler_chose(fake, Q):  # noqa: F811
    """the tile kernel trades the registers of a launch of 96 a thread; with others the call takes passes of eight"""
    cfg = Q.make_q4_cfg(131072, 5120, 128, max_tokens=512)
    a = 1 << 20
    args = [ctypes.byref(cfg), ctypes.c_void_p(a), 512, ctypes.c_int64(5120), *map(ctypes.c_void_p, (a, a, None, a)),
            ctypes.c_int64(131072), ctypes.c_void_p(a), ctypes.c_size_t(1 << 40), None]
    fake.set_registers(88)
    for _ in range(2):
        assert fake.moe_v41_q4_linear(*args) == Q.MOE_OK
        assert counts(fake)[:2] == [64, 0]


@pytest.mark.parametrize("dim,m,streamed", [(5120, 4096, True), (7168, 4096, True), (8192, 153, True), (8192, 152, False),
                                            (8200, 4096, False)])
def test_norm_streams_rows_of_every_width_that_fits(fake, Q, dim, m, streamed):  # noqa: F811
    """f32 rows: more of them than a block each fills the GPU with are streamed, by a few blocks an SM"""
    cfg = Q.make_norm_cfg(dim, y_type=Q.MOE_T_F32, h_type=Q.MOE_T_F32)
    a, d = 1 << 20, ctypes.c_int64(dim)
    p = ctypes.c_void_p
    assert fake.moe_v41_block_norm(ctypes.byref(cfg), m, p(a), d, None, None, None, d, p(a), d, p(a), d, None, None, p(a),
                                   d, None) == Q.MOE_OK
    launches, bad, grid = counts(fake)
    assert launches == 1 and bad == 0
    assert (grid < m) == streamed


# passes of eight tokens, or 1 for the tile kernel: what was the faster of the two when both were measured
@pytest.mark.parametrize("m,n,k,group,launches", [
    (16, 131072, 5120, 128, 2), (17, 131072, 5120, 128, 1), (24, 131072, 5120, 64, 3), (32, 131072, 5120, 64, 1),
    (32, 131072, 5120, 32, 4), (48, 131072, 5120, 32, 1), (9, 5120, 2304, 128, 1), (9, 5120, 2304, 64, 2),
    (24, 5120, 2304, 32, 3), (32, 5120, 2304, 32, 1), (16, 20000, 4096, 32, 2), (32, 20000, 4096, 64, 1),
    (16, 512, 5120, 128, 2), (17, 512, 5120, 128, 1), (32, 4608, 5120, 32, 4), (64, 4608, 5120, 32, 1)])
def test_q4_passes_or_tiles(fake, Q, m, n, k, group, launches):  # noqa: F811
    cfg = Q.make_q4_cfg(n, k, group, max_tokens=m)
    a = 1 << 20
    fake.set_registers(96)
    assert fake.moe_v41_q4_linear(ctypes.byref(cfg), ctypes.c_void_p(a), m, ctypes.c_int64(k),
                                  *map(ctypes.c_void_p, (a, a, None, a)), ctypes.c_int64(n), ctypes.c_void_p(a),
                                  ctypes.c_size_t(1 << 40), None) == Q.MOE_OK
    assert counts(fake)[:2] == [launches, 0]


def test_logprob_bounds_from_pieces_or_threads(fake, Q):  # noqa: F811
    """one kernel for short slices and one for long ones, by what was the faster: f32 from 62 pieces of 4 KB on, 16 bits
    from 97 pieces of 2 KB (many rows: one block a row)"""
    fake.last_kernel.restype = ctypes.c_void_p
    a = ctypes.c_void_p(1 << 20)

    def kernel(vocab, t):
        cfg = Q.make_logprob_cfg(vocab, t, 20)
        assert fake.moe_v41_token_logprobs(ctypes.byref(cfg), a, 1000, ctypes.c_int64(vocab), None, ctypes.c_int64(0),
                                           *[a] * 7, None) == Q.MOE_OK
        return fake.last_kernel()

    for t, short, long in ((Q.MOE_T_F32, (1000, 50000), (64000, 131072)), (Q.MOE_T_BF16, (50001, 65536), (100000, 131072)),
                           (Q.MOE_T_F16, (50001, 65536), (100000, 131072))):
        assert len({kernel(v, t) for v in short}) == 1 and len({kernel(v, t) for v in long}) == 1
        assert kernel(short[0], t) != kernel(long[0], t)


# blocks of whole row tiles of 32 (as many as there are, up to the 152 SMs), or sharing them (152): the faster of the two
@pytest.mark.parametrize("m,n,k,group,grid", [(8, 4608, 5120, 32, 144), (1, 512, 5120, 128, 16), (5, 500, 6144, 128, 16),
                                              (1, 1024, 16384, 128, 152), (2, 700, 20480, 128, 152),
                                              (8, 600, 9216, 128, 152), (1, 512, 32768, 128, 152)])
def test_q4_whole_or_shared_row_tiles(fake, Q, m, n, k, group, grid):  # noqa: F811
    cfg = Q.make_q4_cfg(n, k, group, max_tokens=m)
    a = 1 << 20
    assert fake.moe_v41_q4_linear(ctypes.byref(cfg), ctypes.c_void_p(a), m, ctypes.c_int64(k),
                                  *map(ctypes.c_void_p, (a, a, None, a)), ctypes.c_int64(n), ctypes.c_void_p(a),
                                  ctypes.c_size_t(1 << 40), None) == Q.MOE_OK
    assert counts(fake) == [1, 0, grid]
