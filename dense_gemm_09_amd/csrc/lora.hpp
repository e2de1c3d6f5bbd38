// The low-rank part of a product with adapters: arguments that its kernels take
// next to the product's, and the launch of the first factor's product.
#pragma once

#include <algorithm>

#include "common.hpp"

namespace g355 {

constexpr int kMaxRank = 128;
constexpr int64_t kMaxAdapters = int64_t{1} << 16;

// Rank as the matrix cores take it: a multiple of an MFMA's 16 K elements.
inline int64_t padded_rank(int64_t R) { return (R + 15) / 16 * 16; }

// The first factors' product h[m] = scale[a] * (A[m] down_a) of row m with adapter a.
// It is summed in FP32, over shares of K where that brings more workgroups, and
// multiplied with the second factors as BF16 values whose sum it is (split_h): two for
// BF16 output, off by at most 2^-16 of h, where one value would be off by 2^-8, as much
// as the output's own rounding, before it; three for FP32 output, which hold all of its
// 24 bits. For tiles, which read it often, a row is stored as pad values of each part,
// the highest first; the kernels for few rows add up the shares themselves. Columns from
// the rank on are zeros; rows without an adapter are not written.
constexpr int kMostParts = 3;
inline int parts_of_h(bool f32_out) { return f32_out ? 3 : 2; }

struct LoraShares {
  int shares;
  int len;  // K elements of a share, a multiple of 64
};

// Workgroups that the first factors' product is spread over: one on every CU.
constexpr int64_t kLoraWorkgroups = 256;

inline LoraShares lora_shares(int64_t M, int64_t K, int64_t R) {
  const int64_t units = (M + 15) / 16 * std::max<int64_t>(1, padded_rank(R) / 16);
  const int64_t most = std::min<int64_t>(4, std::max<int64_t>(1, kLoraWorkgroups / units));
  const int64_t shares = std::max<int64_t>(1, std::min(most, (K + 1023) / 1024));
  const int64_t len = std::max<int64_t>(64, ((K + shares - 1) / shares + 63) / 64 * 64);
  return {static_cast<int>(std::max<int64_t>(1, (K + len - 1) / len)), static_cast<int>(len)};
}

struct LoraArgs : GemmArgs {
  const int32_t* adapter;  // INT32[M]
  const uint16_t* h;       // [M][parts * pad], tile kernels
  const float* partial;    // [shares][M][pad], kernels for few rows
  int shares;
  const uint16_t* up;      // adapter g's N rows of rank elements at g * stride_up
  int64_t ld_up, stride_up;
  int adapters;            // G
  int rank, pad;
  int parts;               // of h
};

typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Elements k .. k+7 (k a multiple of 8) of a BF16 row of K at any alignment; zeros
// past its end (what lies there belongs to another row). Without a branch, so that
// loads of many chunks are in flight together: a chunk that the row's end cuts is
// the row's last eight elements shifted, one past it the same made zero. Only rows
// shorter than that are read element by element. In two steps, for loads that are
// to stay in flight: load8_raw, and load8_fix where they are used.
__device__ __forceinline__ i32x4 load8_raw(const uint16_t* row, int k, int K) {
  if (K < 8) {
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 7; ++q)
      if (k + q < K) v[q >> 1] |= static_cast<int>(static_cast<uint32_t>(row[k + q]) << (16 * (q & 1)));
    return v;
  }
  return *reinterpret_cast<const i32x4_any*>(row + min(k, K - 8));
}

__device__ __forceinline__ i32x4 load8_fix(i32x4 v, int k, int K) {
  if (K < 8) return v;
  if ((K & 7) != 0) {  // the same for the whole launch
    i32x4 c = v;       // shifted down by 8 - K % 8 elements
    const int over = 8 - (K & 7);
    if (over & 4) c = i32x4{c[2], c[3], 0, 0};
    if (over & 2) c = i32x4{c[1], c[2], c[3], 0};
    if (over & 1)
      c = i32x4{static_cast<int>(__builtin_amdgcn_alignbyte(c[1], c[0], 2)),
                static_cast<int>(__builtin_amdgcn_alignbyte(c[2], c[1], 2)),
                static_cast<int>(__builtin_amdgcn_alignbyte(c[3], c[2], 2)),
                static_cast<int>(static_cast<uint32_t>(c[3]) >> 16)};
    const bool cut = k + 8 > K;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = cut ? c[q] : v[q];
  }
  const bool in = k < K;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = in ? v[q] : 0;
  return v;
}

__device__ __forceinline__ i32x4 load8(const uint16_t* row, int k, int K) { return load8_fix(load8_raw(row, k, K), k, K); }

// The parts of h (above). Of two, each is rounded to nearest, except that an h which
// BF16 would round to an infinity has its bits cut off; of three, each has its bits cut
// off, so that the last is exact. Infinities and NaN are the highest part's alone.
template <int PARTS>
__device__ __forceinline__ void split_h(float h, uint32_t (&part)[PARTS]) {
  const uint32_t bits = __float_as_uint(h);
  const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
  const uint32_t nearest = f32_to_bf16_bits(h);
  const bool cut = PARTS == 3 || (nearest & 0x7fffu) == 0x7f80u;
  part[0] = finite && cut ? bits >> 16 : nearest;
  float rest = h - bf16_bits_to_f32(static_cast<uint16_t>(part[0]));
  if constexpr (PARTS == 2) {
    part[1] = finite ? f32_to_bf16_bits(rest) : 0u;
  } else {
    part[1] = finite ? __float_as_uint(rest) >> 16 : 0u;
    rest -= bf16_bits_to_f32(static_cast<uint16_t>(part[1]));
    part[2] = finite ? __float_as_uint(rest) >> 16 : 0u;
  }
}

// An infinite second factor times h is an infinity with the sign of both: the highest
// part gives it, and the others, which may be zero or of the other sign, must not turn
// it into NaN. Their products therefore take the factors without their infinities (and
// NaN, which the highest part's product has had as well). unbounded: nonzero if the
// fragment has any; the exponents' carries tell (three instructions for two elements).
__device__ __forceinline__ uint32_t unbounded(const i32x4& v) {
  uint32_t c = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) c |= (static_cast<uint32_t>(v[q]) & 0x7f807f80u) + 0x00800080u;
  return c & 0x80008000u;
}

__device__ __forceinline__ i32x4 bounded(i32x4 v) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t c = ((static_cast<uint32_t>(v[q]) & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    v[q] = static_cast<int>(static_cast<uint32_t>(v[q]) & ~(c | (c - (c >> 15))));
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
  uint16_t* h;         // [M][parts * pad], or nullptr: partial sums are all that is wanted
  float* partial;      // [shares][M][pad] (not used for one share and an h)
  int M, K, adapters, rank, pad, parts;
  int shares, share_len;
  int split;           // workgroups that a tile's adapters are dealt to (set by the launch)
};

hipError_t launch_lora_down(const LoraDownArgs& a, hipStream_t stream);

struct Plan;
struct LaunchSpec;
// The projection's kernel, or its partial sums' (plan.split > 1).
hipError_t launch_lora(const Plan& plan, const LaunchSpec& spec, const LoraArgs& args, hipStream_t stream);
// The same for at most 16 rows (gemm_skinny.hip): operands as for launch_skinny.
hipError_t launch_skinny_lora(const LaunchSpec& spec, const LoraArgs& args, hipStream_t stream);

}  // namespace g355
