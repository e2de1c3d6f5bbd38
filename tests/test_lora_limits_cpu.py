"""Sizes that the projection with adapters refuses before anything is enqueued."""
import pytest

from tests.test_routing_abi_cpu import OK, UNSUP, lora


@pytest.mark.parametrize("ld", [1 << 30, 1 << 32, 1 << 61, 1 << 62, (1 << 62) + 32, (1 << 63) - 1])
@pytest.mark.parametrize("rows", [3, 5, 17, (1 << 30) - 1, 1 << 30])
def test_leading_dimensions_whose_span_exceeds_64_bits(rows, ld):
    """(rows - 1) * ld is beyond 2^31 bytes in all of them, and zero or negative in 64 bits in some."""
    assert lora(M=rows, lda=ld, wsb=1 << 62) == UNSUP
    assert lora(M=200, N=rows, ldb=ld, ldc=1 << 30, wsb=1 << 62) == UNSUP


def test_nothing_to_do_is_not_refused():
    assert lora(M=0, lda=1 << 62) == OK and lora(N=0, ldb=1 << 62) == OK
