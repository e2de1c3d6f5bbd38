// Address arithmetic of the copies of BF16 operands whose rows run along the
// contraction axis (the weight of an input gradient, both operands of a weight
// gradient). Plain constexpr functions, so that the host can call them too.
//
// A slice's copies go through a buffer descriptor whose base is the slice's
// first row. The hardware drops, and reads as zeros, every 4-byte word of a
// 16-byte copy that does not lie wholly inside the descriptor's range.
#pragma once

#include <cstdint>

namespace g355 {

// Offset of a copy that brings zeros: past every range.
constexpr uint32_t kNowhere = 0x80000000u;

// Offset of columns n .. n+7 of row k of a slice; rows are ld2 bytes apart, K in
// all. 64 rows, or all that there are, span less than 2^31 bytes (the host checks
// it), and where K is shorter than a slice the rows past it get no offset: far
// apart, theirs would wrap round to a row that exists.
constexpr uint32_t rows_offset(int k, uint32_t ld2, int n, int cols, int K) {
  return n < cols && k < K ? static_cast<uint32_t>(k) * ld2 + static_cast<uint32_t>(n * 2) : kNowhere;
}

// Most rows of a slice, and the rows from which on no slice needs a limit: a copy in
// row 63 reads at most 7 elements past its row's last, and 8 more rows hold them.
constexpr int kSliceRows = 64;
constexpr int kFreeRows = kSliceRows + 8;

// Range of the descriptor of a slice with `rem` rows up to the end of K, `cols`
// columns from its base. Where the operand ends, the range ends with row
// rem - 1: later rows then read zeros, and a chunk that straddles the last column
// of the last row reads no word past that column (in the rows before, it reads
// what follows the row, into columns that are never stored). For an odd number
// of columns the last word holds the last element and two bytes more, so the
// range is 2 bytes longer (rows_dma_ok: those bytes are on the operand's last
// page). 32 bits, as this is computed for every copy: in 64 bits a weight gradient of
// 16384 rows over 8 experts, 14336 x 4096, takes 1765 us, so 1720.
constexpr int rows_range(int rem, uint32_t ld2, int cols) {
  if (rem >= kFreeRows) return INT32_MAX;
  const uint32_t want = rem > 0 ? static_cast<uint32_t>(rem - 1) * ld2 + static_cast<uint32_t>(cols * 2 + 2) : 0;
  return static_cast<int>(want < INT32_MAX ? want : INT32_MAX);
}

// Whether these copies may take an array at `base`: rows of ld elements (groups
// `stride` apart), its last element `last`. They read up to two bytes past that
// element, in a 4-byte word that holds it: inside the same aligned word where
// every row starts on one, else on the same page unless the array ends with a
// page. Elsewhere operands are loaded through registers.
constexpr bool rows_dma_ok(uintptr_t base, int64_t ld, int64_t stride, int64_t last) {
  if (base & 1u) return false;
  if (base % 4 == 0 && ld % 2 == 0 && stride % 2 == 0) return true;
  return (base + 2 * static_cast<uintptr_t>(last + 1)) % 4096 != 0;
}

}  // namespace g355
