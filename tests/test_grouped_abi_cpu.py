"""Refusals of the INT8 and grouped entry points: all before anything is enqueued, no GPU needed."""
import pytest
import torch

import dense_gemm_09_amd as g
from dense_gemm_09_amd import COL, OUT_BF16, OUT_F32, ROW

OK, NULLP, BAD_DIM, BAD_LD, BAD_ENUM, UNSUP = range(6)
FAKE = 0x7F0000000000


def int8(M=64, N=64, K=64, A=FAKE, lda=None, la=ROW, B=FAKE, ldb=None, lb=COL, sa=FAKE, za=None, sb=FAKE,
         sums=None, C=FAKE, ldc=None, cd=OUT_F32, act=0):
    return g.lib().gemm_int8_scaled(M, N, K, 1.0, A, K if lda is None else lda, la, B,
                                    K if ldb is None else ldb, lb, sa, za, sb, sums, 0.0, C,
                                    N if ldc is None else ldc, cd, None, act, None, 0, None)


def test_int8_refusals():
    assert int8(cd=2) == BAD_ENUM and int8(act=9) == BAD_ENUM and int8(la=3) == BAD_ENUM
    assert int8(M=-1) == BAD_DIM and int8(K=1 << 31) == BAD_DIM
    assert int8(la=COL) == UNSUP and int8(lb=ROW) == UNSUP
    assert int8(K=131072) == UNSUP
    assert int8(lda=63) == BAD_LD and int8(ldb=63) == BAD_LD and int8(ldc=63) == BAD_LD
    for name in ("A", "B", "C", "sa", "sb"):
        assert int8(**{name: None}) == NULLP
    assert int8(za=FAKE) == NULLP and int8(sums=FAKE) == NULLP
    assert int8(M=0) == OK and int8(N=0, ldc=1) == OK


def test_int8_quant_refusals():
    def call(os_=FAKE, oz=None, q=0, Q=FAKE):
        return g.lib().gemm_int8_scaled_quant(8, 8, 8, 1.0, FAKE, 8, ROW, FAKE, 8, COL, FAKE, None, FAKE,
                                              None, None, 0, os_, oz, Q, 8, q, None, 0, None)
    assert call(q=2) == BAD_ENUM and call(os_=None) == NULLP and call(Q=None) == NULLP
    assert call(oz=FAKE, q=1) == UNSUP


def test_quantiser_and_sum_refusals():
    q = g.lib().gemm_quantize_int8_rows
    assert q(-1, 8, FAKE, 8, FAKE, 8, FAKE, None) == BAD_DIM
    assert q(8, 8, FAKE, 7, FAKE, 8, FAKE, None) == BAD_LD
    assert q(8, 8, FAKE, 8, FAKE, 7, FAKE, None) == BAD_LD
    assert q(8, 8, None, 8, FAKE, 8, FAKE, None) == NULLP
    assert q(8, 8, FAKE, 8, FAKE, 8, None, None) == NULLP
    assert q(0, 8, None, 8, None, 8, None, None) == OK
    s = g.lib().gemm_int8_col_sums
    assert s(8, -1, FAKE, 8, FAKE, None) == BAD_DIM
    assert s(131072, 8, FAKE, 131072, FAKE, None) == UNSUP
    assert s(8, 8, FAKE, 7, FAKE, None) == BAD_LD
    assert s(8, 8, None, 8, FAKE, None) == NULLP and s(8, 8, FAKE, 8, None, None) == NULLP
    assert s(8, 0, None, 8, None, None) == OK


def bf16(G=4, T=64, N=64, K=64, A=FAKE, lda=None, off=FAKE, B=FAKE, ldb=None, lb=COL, stride=4096, C=FAKE,
         ldc=None, cd=OUT_F32, act=0):
    return g.lib().gemm_grouped_bf16(G, T, N, K, 1.0, A, K if lda is None else lda, off, B,
                                     (K if lb == COL else N) if ldb is None else ldb, lb, stride, 0.0, C,
                                     N if ldc is None else ldc, cd, None, act, None)


def scaled(fn, layout=COL, sa=FAKE, sb=FAKE, K=64, zeros=()):
    return getattr(g.lib(), fn)(4, 64, 64, K, 1.0, FAKE, K, FAKE, FAKE, max(K, 64), layout, 4096, sa, *zeros[:1],
                                sb, *zeros[1:], 0.0, FAKE, 64, OUT_BF16, None, 0, None)


def test_grouped_refusals():
    assert bf16(lb=2) == BAD_ENUM and bf16(cd=3) == BAD_ENUM and bf16(act=-1) == BAD_ENUM
    for name in ("G", "T", "N", "K"):
        assert bf16(**{name: -1}) == BAD_DIM
    assert bf16(G=65537) == BAD_DIM and bf16(T=(1 << 30) + 1) == BAD_DIM
    assert bf16(T=1 << 30, N=1 << 30, ldc=1 << 30) == BAD_DIM  # more workgroups than a grid has
    assert bf16(lda=63) == BAD_LD and bf16(ldb=63) == BAD_LD and bf16(ldc=63) == BAD_LD
    assert bf16(lb=ROW, ldb=63) == BAD_LD and bf16(stride=-1) == BAD_LD
    for name in ("A", "B", "C", "off"):
        assert bf16(**{name: None}) == NULLP
    assert bf16(off=FAKE + 2) == UNSUP
    assert bf16(G=0) == OK and bf16(T=0, A=None) == OK and bf16(N=0, ldc=1) == OK


@pytest.mark.parametrize("fn", ["gemm_grouped_fp8_scaled", "gemm_grouped_int8_scaled"])
def test_grouped_8bit_refusals(fn):
    zeros = (None, None) if "int8" in fn else ()
    assert scaled(fn, ROW, zeros=zeros) == UNSUP
    assert scaled(fn, sa=None, zeros=zeros) == NULLP and scaled(fn, sb=None, zeros=zeros) == NULLP
    if zeros:
        assert scaled(fn, K=131072, zeros=zeros) == UNSUP
        assert scaled(fn, zeros=(FAKE, None)) == NULLP and scaled(fn, zeros=(None, FAKE)) == NULLP


def wgrad(G=4, T=64, N=32, K=48, D=FAKE, ldd=None, X=FAKE, ldx=None, off=FAKE, C=FAKE, ldc=None,
          stride=None, cd=OUT_F32):
    ldc = K if ldc is None else ldc
    return g.lib().gemm_grouped_bf16_wgrad(G, T, N, K, 1.0, D, N if ldd is None else ldd, X,
                                           K if ldx is None else ldx, off, 0.0, C, ldc,
                                           N * ldc if stride is None else stride, cd, None)


def test_wgrad_refusals():
    assert wgrad(cd=2) == BAD_ENUM
    for name in ("G", "T", "N", "K"):
        assert wgrad(**{name: -1}) == BAD_DIM
    assert wgrad(ldd=31) == BAD_LD and wgrad(ldx=47) == BAD_LD and wgrad(ldc=47) == BAD_LD
    assert wgrad(stride=31 * 48 + 47) == BAD_LD  # one group's gradient would overlap the next
    for name in ("D", "X", "C", "off"):
        assert wgrad(**{name: None}) == NULLP
    assert wgrad(off=FAKE + 1) == UNSUP
    assert wgrad(G=0) == OK and wgrad(N=0, ldd=1, stride=0) == OK
    assert wgrad(K=0, ldx=1, ldc=1, stride=0) == OK


def test_python_checks_the_bytes_each_call_touches():
    """Host tensors are refused before the library is reached."""
    t = torch.zeros(64 * 64, dtype=torch.int8)
    f = torch.zeros(64)
    with pytest.raises(ValueError, match="A must be a device tensor"):
        g.gemm_int8_scaled(64, 64, 64, 1.0, t, 64, ROW, t, 64, COL, f, None, f, None, 0.0, f, 64, OUT_F32)
    with pytest.raises(ValueError, match="X must be a device tensor"):
        g.quantize_int8_rows(4, 8, torch.zeros(32, dtype=torch.bfloat16), 8, t, 8, f)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="A must be a device tensor"):
        g.gemm_grouped_bf16(2, 4, 8, 8, 1.0, t, 8, off, t, 8, COL, 64, 0.0, f, 8, OUT_F32)
    with pytest.raises(ValueError, match="D must be a device tensor"):
        g.gemm_grouped_bf16_wgrad(2, 4, 8, 8, 1.0, t, 8, t, 8, off, 0.0, f, 8, 64, OUT_F32)
