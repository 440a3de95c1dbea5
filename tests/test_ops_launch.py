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
