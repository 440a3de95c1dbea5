"""The attention block's launchers without a GPU: the library's objects linked with
a runtime that launches nothing (fake_cudart.cc)."""
import ctypes
import os
import subprocess
import threading

import pytest
from test_attn_args import A, Q, _attn, _kv, _seqs  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture
def fake(Q, tmp_path):  # noqa: F811
    lib_dir = os.path.dirname(Q.SO)
    objs = [os.path.join(lib_dir, f"{o}.o") for o in ("k_rope", "k_attn_rows", "k_attn_tiles", "attn_launch", "attn_capi",
                                                      "k_logprob", "k_norm", "k_q4", "k_q4_gemm", "ops_capi")]
    so = str(tmp_path / "fake.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", "/usr/local/cuda/include", "-Wl,-Bsymbolic",
                    os.path.join(HERE, "fake_cudart.cc"), *objs, "-o", so, "-lpthread"], check=True)
    lib = ctypes.CDLL(so)
    lib.last_kernel.restype = ctypes.c_void_p
    lib.set_registers(168)
    return lib


def counts(lib):
    out = (ctypes.c_int * 3)()
    lib.counts(out)
    return list(out)


def attend(fake, Q, cfg, m, new, batch=3):  # noqa: F811
    a, seqs = ctypes.c_void_p(A), _seqs(Q, batch=batch)
    row = ctypes.c_int64(cfg.heads * cfg.kv.head_dim)
    rc = fake.moe_v41_paged_attention(ctypes.byref(cfg), ctypes.byref(seqs), m, new, a, row, a, a, a, row, a,
                                      ctypes.c_int64(cfg.heads), a, ctypes.c_size_t(1 << 40), None)
    return rc, fake.last_kernel()


# up to 16 rows (tokens of a sequence x heads of a group): the kernel for few rows; above, the one for many
@pytest.mark.parametrize("heads,kv_heads,few,many", [(8, 8, 16, 17), (32, 8, 4, 5), (40, 8, 3, 4), (64, 4, 1, 2),
                                                     (128, 4, 0, 1)])
def test_rows_choose_the_kernel(fake, Q, heads, kv_heads, few, many):  # noqa: F811
    cfg = Q.make_attn_cfg(_kv(Q, kv_heads=kv_heads), heads)
    assert attend(fake, Q, cfg, 5, few)[0] == Q.MOE_OK
    rows = attend(fake, Q, cfg, 5, few)[1]
    assert attend(fake, Q, cfg, 5, 0) == (Q.MOE_OK, rows)
    tiles = attend(fake, Q, cfg, 5, many)[1]
    assert tiles != rows and attend(fake, Q, cfg, 500, 1 << 30) == (Q.MOE_OK, tiles)
    launches, bad, grid = counts(fake)
    assert (launches, bad, grid) == (5, 0, 152)                    # one launch a call, a block an SM


def test_another_number_of_registers_leaves_the_call_to_the_other_kernel(fake, Q):  # noqa: F811
    """the kernel for many rows trades the registers of a launch of 168 a thread"""
    cfg = Q.make_attn_cfg(_kv(Q), 4)
    rows = attend(fake, Q, cfg, 5, 1)[1]
    fake.set_registers(160)
    assert attend(fake, Q, cfg, 5, 100) == (Q.MOE_OK, rows)


def test_types_and_widths_have_their_own_kernels(fake, Q):  # noqa: F811
    seen = set()
    for new in (1, 100):
        for dim in (64, 128):
            for t in (Q.MOE_T_BF16, Q.MOE_T_F16):
                cfg = Q.make_attn_cfg(Q.make_kv_cfg(2, dim, 16, 40, t), 4)
                seen.add(attend(fake, Q, cfg, 5, new)[1])
    assert len(seen) == 8


def test_calls_from_many_threads(fake, Q):  # noqa: F811
    cfgs = [Q.make_attn_cfg(_kv(Q, head_dim=d), 4) for d in (64, 128)]
    bad = []

    def run(i):
        for j in range(300):
            if attend(fake, Q, cfgs[(i + j) % 2], 5, 1 + 99 * (j % 2))[0] != Q.MOE_OK:
                bad.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and counts(fake)[:2] == [1800, 0]


@pytest.mark.parametrize("m,heads,dim,rot", [(1, 1, 2, 2), (1, 32, 128, 128), (1, 65536, 8, 8), (3, 4096, 1024, 1024),
                                             (8192, 32, 128, 64), ((1 << 24) - 1, 1, 16, 16), (5, 3, 7, 4)])
def test_rope_launches_once(fake, Q, m, heads, dim, rot):  # noqa: F811
    a, p = ctypes.c_void_p(A), ctypes.c_int64
    cfg = Q.make_rope_cfg(dim, rot)
    assert fake.moe_v41_rope(ctypes.byref(cfg), m, heads, a, p(heads * dim), p(dim), a, a, ctypes.c_void_p(2 * A),
                             p(heads * dim), p(dim), None) == Q.MOE_OK
    assert counts(fake)[:2] == [1, 0]


def test_append_launches_once(fake, Q):  # noqa: F811
    a, p = ctypes.c_void_p(A), ctypes.c_int64
    rope = Q.make_rope_cfg(64)
    for m in (1, 700, 100000):
        seqs, kv = _seqs(Q), _kv(Q)
        assert fake.moe_v41_kv_append(ctypes.byref(kv), ctypes.byref(rope), ctypes.byref(seqs), m, a, p(128), a, p(128), a, a, 4,
                                      a, p(256), a, p(256), a, None, a, None) == Q.MOE_OK
    assert counts(fake)[:2] == [3, 0]
