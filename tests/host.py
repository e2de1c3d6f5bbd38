"""The library's host arithmetic as a shared library of its own (tests/host_arith.cpp)."""
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        so = os.path.join(d, "host_arith.so")
        r = subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC",
                            "-I", os.path.join(ROOT, "dense_gemm_09_amd", "csrc"),
                            os.path.join(ROOT, "tests", "host_arith.cpp"), "-o", so],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        L = ctypes.CDLL(so)
    i, q = ctypes.c_int, ctypes.c_int64
    L.check_slice.argtypes = [i, i, i, q, i, q]
    L.grouped_tile.argtypes = [q, q, q, i]
    L.wgrad_tile.argtypes = [q, q, q]
    return L
