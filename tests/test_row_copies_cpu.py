"""What the copies of BF16 rows along the contraction axis may read, from their address arithmetic (no GPU).

A slice of 64 rows is copied in 16-byte chunks; the last chunk of a row straddles its last column
where the column count is no multiple of 8, and what it reads past the last row must stay inside the
word of the last element.
"""
import pytest

from tests import host

OVER_READ, LOST, NOT_ZERO, NEXT_PAGE = 1, 2, 4, 8


def check(rem, ld, cols, base=0):
    # As the first slice, and as a later one of an operand whose first 64 rows lie within 2^31 bytes.
    for K in (rem, rem + 64) if 128 * ld < 1 << 31 else (rem,):
        bad = host.lib().check_slice(64, rem, K, ld, cols, base)
        names = [n for n, b in (("reads past the operand", 1), ("loses an element", 2),
                                ("reads rows past the last", 4), ("reads the next page", 8)) if bad & b]
        assert not bad, f"rem={rem} K={K} ld={ld} cols={cols} base={base}: {', '.join(names)}"


@pytest.mark.parametrize("rem", [0, 1, 2, 31, 63, 64, 65, 66, 71, 72, 73, 127, 128, 129, 1000])
def test_a_slice_reads_its_operand_and_nothing_after_it(rem):
    for cols in [*range(1, 26), 127, 128, 255, 256]:
        for pad in (0, 1, 2, 3, 7, 8, 250):
            check(rem, cols + pad, cols)


@pytest.mark.parametrize("rem", [1, 63, 64, 65, 128])
@pytest.mark.parametrize("cols", [1, 2, 5, 6, 241, 252, 255, 256])
def test_an_array_that_ends_with_a_page_or_near_one(rem, cols):
    for ld in (cols, cols + 1, cols + 2):
        size = 2 * ((rem - 1) * ld + cols)
        for past in range(-6, 8, 2):  # where the array ends, from a page's end on
            check(rem, ld, cols, (past - size) % 4096)


def test_long_and_far_apart_rows():
    """Ranges past 2^31 bytes: the operand goes on after the slice."""
    for ld in (1 << 20, (1 << 23) + 3, (1 << 24) - 8):
        for rem in (1, 64, 65, 1000):
            check(rem, ld, 255)


def test_few_rows_far_apart():
    """Rows of the slice past the operand's last, whose offsets pass 32 bits, bring zeros."""
    for rem, ld in ((2, 1 << 29), (1, (1 << 31) - 1), (5, (1 << 26) + 1), (8, 1 << 26), (33, (1 << 24) + 2)):
        for cols in (1, 9, 256):
            check(rem, ld, cols)
