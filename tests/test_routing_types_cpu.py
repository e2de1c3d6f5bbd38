"""Matrices of another type than the call says are refused by the binding: their bytes would be read as other numbers.

Host tensors suffice: the type is looked at first. What passes is refused for being on the host, or, as an address,
goes on to the library's own checks."""
import pytest
import torch

import dense_gemm_09_amd as g
from dense_gemm_09_amd import OUT_BF16, OUT_F32

FAKE = 0x7F0000000000
KINDS = {OUT_F32: torch.float32, OUT_BF16: torch.bfloat16}
ALL = [torch.float16, torch.float32, torch.bfloat16, torch.float64, torch.int32, torch.int16, torch.uint8]


def route(x, kind):
    g.route(2, 8, 2, x, 8, kind, g.SCORE_SOFTMAX, None, 1, 1, 1, False, 1.0, FAKE, FAKE)


def grad(x, kind):
    g.route_grad(2, 8, 2, x, 8, kind, g.SCORE_SOFTMAX, False, 1.0, FAKE, FAKE, FAKE, 8)


def dlogits(x, kind):
    g.route_grad(2, 8, 2, FAKE, 8, kind, g.SCORE_SOFTMAX, False, 1.0, FAKE, FAKE, x, 8)


def combine_y(x, kind):
    g.combine_rows(2, 2, 4, 8, x, 8, kind, FAKE, None, 0.0, FAKE, 8, OUT_F32)


def combine_c(x, kind):
    g.combine_rows(2, 2, 4, 8, FAKE, 8, OUT_F32, FAKE, None, 0.0, x, 8, kind)


def grad_d(x, kind):
    g.combine_rows_grad(2, 2, 4, 8, x, 8, kind, FAKE, 8, OUT_F32, FAKE, None, FAKE, 8, FAKE)


def grad_y(x, kind):
    g.combine_rows_grad(2, 2, 4, 8, FAKE, 8, OUT_F32, x, 8, kind, FAKE, None, FAKE, 8, FAKE)


def grad_dy(x, kind):
    g.combine_rows_grad(2, 2, 4, 8, FAKE, 8, OUT_F32, FAKE, 8, kind, FAKE, None, x, 8, FAKE)


def lora(**kw):
    v = dict(A=FAKE, B=FAKE, down=FAKE, up=FAKE, C=FAKE, bias=FAKE, kind=OUT_F32)
    v.update(kw)
    g.gemm_lora_bf16(2, 8, 8, 2, 4, 1.0, v["A"], 8, v["B"], 8, FAKE, v["down"], 8, 32, v["up"], 4, 32, None, 0.0, v["C"],
                     8, v["kind"], v["bias"])


@pytest.mark.parametrize("call", [route, grad, dlogits, combine_y, combine_c, grad_d, grad_y, grad_dy,
                                  lambda x, kind: lora(C=x, kind=kind)])
@pytest.mark.parametrize("kind", [OUT_F32, OUT_BF16])
@pytest.mark.parametrize("dtype", ALL)
def test_types(call, kind, dtype):
    x = torch.zeros(256, dtype=dtype)
    match = "must be a device tensor" if dtype in (KINDS[kind], torch.uint8) else \
        f"must be {'FP32' if kind == OUT_F32 else 'BF16'}, not {dtype}"
    with pytest.raises(ValueError, match=match):
        call(x, kind)


@pytest.mark.parametrize("name", ["A", "B", "down", "up", "bias"])
@pytest.mark.parametrize("dtype", ALL)
def test_operands_of_adapters(name, dtype):
    match = "must be a device tensor" if dtype in (torch.bfloat16, torch.uint8) else f"{name} must be BF16, not {dtype}"
    with pytest.raises(ValueError, match=match):
        lora(**{name: torch.zeros(256, dtype=dtype)})


@pytest.mark.parametrize("elem", [1, 2, 4])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.float16, torch.bfloat16, torch.float32, torch.float64])
def test_dispatch_moves_elements_of_the_size_it_is_told(dtype, elem):
    x = torch.zeros(256, dtype=dtype)
    match = "must be a device tensor" if x.element_size() in (1, elem) else "elements have"
    with pytest.raises(ValueError, match=match):
        g.dispatch_rows(2, 2, 4, 8, x, 8, elem, FAKE, FAKE, 8)
    with pytest.raises(ValueError, match=match):
        g.dispatch_rows(2, 2, 4, 8, FAKE, 8, elem, FAKE, x, 8)
