// The library's host arithmetic (copy addresses, grouped plans) for the tests: compiled with g++.
#include <cstring>

#include "grouped_plan.hpp"
#include "row_copies.hpp"

using namespace g355;

namespace {

// What a copy's descriptor lets through, as the hardware does it: 4-byte words
// wholly inside the range. Word w of the 16 bytes at `off`.
bool admitted(uint32_t off, int w, int range) {
  return static_cast<int64_t>(off) + 4 * w + 4 <= static_cast<int64_t>(static_cast<uint32_t>(range));
}

enum : int { OVER_READ = 1, LOST = 2, NOT_ZERO = 4, NEXT_PAGE = 8 };

}  // namespace

extern "C" {

// The copies of one slice of an operand of `cols` columns and K rows, whose first
// row is at byte `base` (mod 4096): `rows` rows of the slice's place in LDS, `rem` rows
// of the operand from the slice on. Returns a set of: a word more than 2 bytes past the last element is
// read; an element is not; an element of a row past `rem` is; a byte on the
// page after the last element's is read although rows_dma_ok admits the array.
int check_slice(int rows, int rem, int K, int64_t ld, int cols, int64_t base) {
  int bad = 0;
  const int64_t ld2 = 2 * ld;
  const int range = rows_range(rem, static_cast<uint32_t>(ld2), cols);
  const int64_t end = rem > 0 ? (rem - 1) * ld2 + 2 * cols : 0;  // bytes up to and with the last element
  const bool ok = rows_dma_ok(static_cast<uintptr_t>(base), ld, 0, rem > 0 ? end / 2 - 1 : 0);
  for (int k = 0; k < rows; ++k) {
    for (int n = 0; n < (cols + 15) / 8 * 8; n += 8) {
      const uint32_t off = rows_offset(k, static_cast<uint32_t>(ld2), n, cols, K);
      for (int w = 0; w < 4; ++w) {
        const bool in = admitted(off, w, range);
        const int64_t to = static_cast<int64_t>(off) + 4 * w + 4;
        if (in && to > end + 2) bad |= OVER_READ;
        if (in && ok && (base + to - 1) / 4096 > (base + end - 1) / 4096) bad |= NEXT_PAGE;
        for (int e = 0; e < 2; ++e) {
          const bool element = n + 2 * w + e < cols;
          const bool here = in && static_cast<int64_t>(off) == k * ld2 + 2 * n;
          if (element && k < rem && !here) bad |= LOST;
          if (element && k >= rem && in) bad |= NOT_ZERO;
        }
      }
    }
  }
  return bad;
}

int grouped_tile(int64_t G, int64_t T, int64_t N, int b_rows) { return plan_grouped(G, T, N, b_rows != 0).bm; }
int wgrad_tile(int64_t G, int64_t N, int64_t K) { return plan_wgrad(G, N, K).bm; }

}  // extern "C"
