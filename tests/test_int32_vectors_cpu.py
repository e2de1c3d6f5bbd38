"""Integer vectors of another type are refused: read as INT32, an INT64 tensor (what cumsum and sum give) has
enough bytes and means something else. Operands are addresses here, which the binding does not look into."""
import pytest
import torch

import dense_gemm_09_amd as g
from dense_gemm_09_amd import COL, OUT_F32, QOUT_INT8, ROW

PTR = 0x7F0000000000


def grouped(offsets):
    g.gemm_grouped_bf16(2, 8, 8, 8, 1.0, PTR, 8, offsets, PTR, 8, COL, 64, 0.0, PTR, 8, OUT_F32)


def grouped_fp8(offsets):
    g.gemm_grouped_fp8_scaled(2, 8, 8, 8, 1.0, PTR, 8, offsets, PTR, 8, COL, 64, PTR, PTR, 0.0, PTR, 8, OUT_F32)


def grouped_int8(offsets=PTR, zero_a=PTR, sum_b=PTR):
    g.gemm_grouped_int8_scaled(2, 8, 8, 8, 1.0, PTR, 8, offsets, PTR, 8, COL, 64, PTR, zero_a, PTR, sum_b, 0.0, PTR,
                               8, OUT_F32)


def wgrad(offsets):
    g.gemm_grouped_bf16_wgrad(2, 8, 8, 8, 1.0, PTR, 8, PTR, 8, offsets, 0.0, PTR, 8, 64, OUT_F32)


def int8(zero_a=PTR, sum_b=PTR):
    g.gemm_int8_scaled(8, 8, 8, 1.0, PTR, 8, ROW, PTR, 8, COL, PTR, zero_a, PTR, sum_b, 0.0, PTR, 8, OUT_F32)


def int8_quant(zero_a=PTR, sum_b=PTR, out_zero=PTR):
    g.gemm_int8_scaled_quant(8, 8, 8, 1.0, PTR, 8, ROW, PTR, 8, COL, PTR, zero_a, PTR, sum_b, None, 0, PTR, out_zero,
                             PTR, 8, QOUT_INT8)


def col_sums(sums):
    g.int8_col_sums(8, 8, PTR, 8, sums)


@pytest.mark.parametrize("dtype", [torch.int64, torch.int16, torch.float32, torch.float64])
@pytest.mark.parametrize("call,name", [(grouped, "offsets"), (grouped_fp8, "offsets"), (grouped_int8, "offsets"),
                                       (grouped_int8, "zero_a"), (grouped_int8, "sum_b"), (wgrad, "offsets"),
                                       (int8, "zero_a"), (int8, "sum_b"), (int8_quant, "zero_a"),
                                       (int8_quant, "sum_b"), (int8_quant, "out_zero"), (col_sums, "sums")])
def test_refused(call, name, dtype):
    with pytest.raises(ValueError, match=f"{name} must be INT32"):
        call(**{name: torch.zeros(64, dtype=dtype)})
    with pytest.raises(ValueError, match=f"{name} must be a device tensor"):
        call(**{name: torch.zeros(64, dtype=torch.int32)})
