// Division of the order of rows by expert into workgroups. Host arithmetic only,
// without HIP.
#pragma once

#include <algorithm>
#include <cstdint>

namespace g355 {

constexpr int kMaxOrderGroups = 8192;  // counters of a workgroup in LDS

// Sorted by one workgroup, which holds the slots' experts in registers and its 16
// waves' counters in LDS.
constexpr int kSmallSlots = 8192;
constexpr int kSmallGroups = 2047;
inline bool order_small(int64_t S, int64_t G) { return S <= kSmallSlots && G <= kSmallGroups; }

constexpr int kSmallWaves = 16;  // 512 slots a wave, eight to a lane
constexpr int kOrderWaves = 4;
constexpr int kHeldKeys = 8;     // keys that a lane holds at a time
constexpr int kMaxChunks = 128;

// The division of S slots into chunks, each a multiple of 64 slots per wave. No slots
// are no chunks, except that the one workgroup's form always has one.
inline void order_chunks(int64_t S, int64_t G, int& chunk, int& chunks) {
  if (order_small(S, G)) {
    chunk = static_cast<int>((S + 64 * kSmallWaves - 1) / (64 * kSmallWaves) * (64 * kSmallWaves));
    chunks = 1;
    return;
  }
  const int64_t least = 64 * kHeldKeys * kOrderWaves;
  const int64_t per = std::max<int64_t>(1, (S + kMaxChunks - 1) / kMaxChunks);
  chunk = static_cast<int>((per + least - 1) / least * least);
  chunks = static_cast<int>((S + chunk - 1) / chunk);
}

}  // namespace g355
