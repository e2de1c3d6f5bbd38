// The low-rank part of a product with adapters: arguments that its kernels take
// next to the product's, and the launch of the first factor's product.
#pragma once

#include "common.hpp"

namespace g355 {

constexpr int kMaxRank = 128;
constexpr int64_t kMaxAdapters = int64_t{1} << 16;

// Rank as the matrix cores take it: a multiple of an MFMA's 16 K elements.
inline int64_t padded_rank(int64_t R) { return (R + 15) / 16 * 16; }

// H holds, for row m with adapter a, h = scale[a] * (A[m] down_a) as two BF16
// values: pad high parts RNE(h), then pad low parts RNE(h - high). h is off by
// at most 2^-16 of itself, where one BF16 value would be off by 2^-8: as much as
// the output's own rounding, before it. Columns from the rank on are zeros, and so
// are rows without an adapter.
struct LoraArgs : GemmArgs {
  const int32_t* adapter;  // INT32[M]
  uint16_t* h;             // [M][2 * pad]
  const uint16_t* up;      // adapter g's N rows of rank elements at g * stride_up
  int64_t ld_up, stride_up;
  int adapters;            // G
  int rank, pad;
};

typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Elements k .. k+7 of a BF16 row of K at any alignment; zeros past its end (what lies
// there belongs to another row).
__device__ __forceinline__ i32x4 load8(const uint16_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 8 <= K) {
    v = *reinterpret_cast<const i32x4_any*>(row + k);
  } else if (k < K) {
#pragma unroll
    for (int q = 0; q < 7; ++q)
      if (k + q < K) v[q >> 1] |= static_cast<int>(static_cast<uint32_t>(row[k + q]) << (16 * (q & 1)));
  }
  return v;
}

struct LoraDownArgs {
  const uint16_t* A;
  int64_t lda;
  const int32_t* adapter;
  const uint16_t* down;
  int64_t ld_down, stride_down;
  const float* scale;  // or nullptr: ones
  uint16_t* h;
  int M, K, adapters, rank, pad;
};

hipError_t launch_lora_down(const LoraDownArgs& a, hipStream_t stream);

struct Plan;
struct LaunchSpec;
// The projection's kernel, or its partial sums' (plan.split > 1).
hipError_t launch_lora(const Plan& plan, const LaunchSpec& spec, const LoraArgs& args, hipStream_t stream);

}  // namespace g355
