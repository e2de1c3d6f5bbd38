"""The division of the order of rows by expert into workgroups (csrc/order_plan.hpp), on the host."""
import os
import subprocess
import sys

import pytest

from tests.host import ROOT

RUN = """
import ctypes, sys
L = ctypes.CDLL(sys.argv[1])
q = ctypes.c_int64
L.order_division.argtypes = [q, q, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
a, b = ctypes.c_int(), ctypes.c_int()
L.order_division(int(sys.argv[2]), int(sys.argv[3]), a, b)
print(a.value, b.value, L.order_is_small(q(int(sys.argv[2])), q(int(sys.argv[3]))))
"""


@pytest.fixture(scope="module")
def so(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("order") / "order_arith.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "dense_gemm_09_amd", "csrc"),
                    os.path.join(ROOT, "tests", "order_arith.cpp"), "-o", out], check=True)
    return out


def division(so, S, G):
    # In a process of its own: a division by zero ends it.
    r = subprocess.run([sys.executable, "-c", RUN, so, str(S), str(G)], capture_output=True, text=True)
    assert r.returncode == 0, (S, G, r.returncode)
    return map(int, r.stdout.split())


@pytest.mark.parametrize("G", [0, 1, 2047, 2048, 8192])
@pytest.mark.parametrize("S", [0, 1, 2048, 8192, 8193, 1 << 18, (1 << 18) + 1, 1 << 30])
def test_division(so, S, G):
    chunk, chunks, small = division(so, S, G)
    if small:
        assert chunks == 1 and chunk >= S and chunk % 1024 == 0
        return
    # Whole segments of waves; no chunk without slots, so that no slots are no chunks.
    assert chunk > 0 and chunk % 256 == 0 and chunks <= 128
    assert chunks * chunk >= S and (chunks - 1) * chunk < max(S, 1)
    assert (chunks == 0) == (S == 0)
