// Per-token FP8 quantisation of BF16 activations: the step that produces the
// FP8 GEMM's A operand and its per-row scales.
//
// The FP8 DeepGEMM page (sec. 1.2) pairs E4M3 activations with one scale per
// token and observes that scale handling done in separate kernels costs extra
// launches and extra trips through memory. Here one workgroup owns one row and
// produces its scale and its codes in a single launch, reading the row from
// HBM once:
//
//   scale[m] = fp32(amax_k |x(m,k)| / 448)      (1 for an all-zero row)
//   Q[m, k]  = E4M3 code of RNE(x(m,k) / scale[m]), saturating at +-448
//
// The division is IEEE float32 division (correctly rounded), so the quotient
// that decides each code is the same float32 value any IEEE implementation
// computes; the float32 -> E4M3 step is gfx950's v_cvt_pk_fp8_f32 (round to
// nearest even) after clamping to +-448. |x| / scale exceeds 448 by at most a
// rounding error, so the clamp only ever maps such values to 448.
//
// One wave owns one row. A row of up to 4096 elements is loaded once into
// registers (all of a lane's loads issued before any is used), reduced to its
// amax with cross-lane shuffles, and encoded from the registers; longer rows
// re-read their tail from cache. HBM traffic is 2 bytes read + 1 byte written
// per element. The register-held part is read and written non-temporally
// (touched once; 14-20% faster than cached accesses at 4096 x 2048 and
// 8192 x 4096).

#include "common.hpp"
#include "internal.hpp"

namespace g355 {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kQuantThreads = 256;   // four waves, one row each
constexpr int kChunk = 512;          // elements of a row one wave covers per 16-byte load
constexpr int kCached = 8;           // chunks kept in registers (rows up to 4096 elements)

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

__device__ __forceinline__ float amax8(float amax, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    amax = fmaxf(amax, fabsf(__uint_as_float(w[j] << 16)));
    amax = fmaxf(amax, fabsf(__uint_as_float(w[j] & 0xffff0000u)));
  }
  return amax;
}

__device__ __forceinline__ uint2 codes8(const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16) / s;
    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) / s;
  }
  return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
}

// One wave per row. VEC: 16-byte loads of 8 BF16 and 8-byte stores of 8
// codes; the first kCached chunks of the row are loaded up front and kept in
// registers for the second pass (longer rows re-read the rest, from cache);
// otherwise element by element.
template <bool VEC>
__global__ void __launch_bounds__(kQuantThreads)
quantize_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, uint8_t* __restrict__ Q,
                     int64_t ldq, float* __restrict__ scale, int M, int K) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.x * (kQuantThreads / 64) + (threadIdx.x >> 6);
  if (m >= M) return;  // no barrier below: a wave may leave early
  const uint16_t* x = X + static_cast<int64_t>(m) * ldx;
  uint8_t* q = Q + static_cast<int64_t>(m) * ldq;

  float amax = 0.f;
  if constexpr (VEC) {
    uint4 c[kCached];
#pragma unroll
    for (int ch = 0; ch < kCached; ++ch) {
      const int k = ch * kChunk + 8 * lane;
      c[ch] = make_uint4(0u, 0u, 0u, 0u);
      if (k < K) {
        const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + k));
        c[ch] = make_uint4(t[0], t[1], t[2], t[3]);
      }
    }
#pragma unroll
    for (int ch = 0; ch < kCached; ++ch) amax = amax8(amax, c[ch]);
    for (int k = kCached * kChunk + 8 * lane; k < K; k += kChunk)
      amax = amax8(amax, *reinterpret_cast<const uint4*>(x + k));
    amax = wave_max(amax);
    const float s = amax > 0.f ? amax / 448.f : 1.f;
    if (lane == 0) scale[m] = s;
#pragma unroll
    for (int ch = 0; ch < kCached; ++ch) {
      const int k = ch * kChunk + 8 * lane;
      if (k < K) {
        const uint2 w = codes8(c[ch], s);
        __builtin_nontemporal_store(u32x2{w.x, w.y}, reinterpret_cast<u32x2*>(q + k));
      }
    }
    for (int k = kCached * kChunk + 8 * lane; k < K; k += kChunk)
      *reinterpret_cast<uint2*>(q + k) = codes8(*reinterpret_cast<const uint4*>(x + k), s);
  } else {
    for (int k = lane; k < K; k += 64) amax = fmaxf(amax, fabsf(bf16_bits_to_f32(x[k])));
    amax = wave_max(amax);
    const float s = amax > 0.f ? amax / 448.f : 1.f;
    if (lane == 0) scale[m] = s;
    for (int k = lane; k < K; k += 64) {
      const float y = bf16_bits_to_f32(x[k]) / s;
      q[k] = static_cast<uint8_t>(e4m3x4(y, 0.f, 0.f, 0.f) & 0xffu);
    }
  }
}

// ------------------------------------------------------------------ INT8 rows

// Per-token INT8 quantisation, the A operand and scale_a of the INT8 product:
//   scale[m] = fp32(amax_k |x(m,k)| / 127)     (1 for an all-zero row)
//   Q[m, k]  = RNE(fp32(x(m,k) / scale[m])) in [-127, 127]
// with IEEE division, as above: the quotient decides the code.
//
// W waves own a row (1 or 4): each lane keeps up to kCached 16-byte loads of it
// in registers, so rows up to W * 4096 elements are read from HBM once and
// from no cache after. One barrier joins the waves' maxima.

// Eight codes of the elements in v.
__device__ __forceinline__ uint2 int8_codes8(const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = quant_i8(__uint_as_float(w[j] << 16) / s, 1.f, 0.f);
    const uint32_t hi = quant_i8(__uint_as_float(w[j] & 0xffff0000u) / s, 1.f, 0.f);
    out[j >> 1] |= (lo | (hi << 8)) << (16 * (j & 1));
  }
  return make_uint2(out[0], out[1]);
}

template <int W, bool VEC>
__global__ void __launch_bounds__(kQuantThreads)
quantize_int8_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, uint8_t* __restrict__ Q,
                          int64_t ldq, float* __restrict__ scale, int M, int K) {
  constexpr int ROWS = kQuantThreads / 64 / W;  // rows per workgroup
  constexpr int T = 64 * W;                     // threads per row
  __shared__ float part[kQuantThreads / 64];
  const int t = threadIdx.x % T;
  const int m = blockIdx.x * ROWS + threadIdx.x / T;
  const bool live = m < M;  // with W = 1 the last workgroup's spare waves have no row
  const uint16_t* x = X + static_cast<int64_t>(live ? m : 0) * ldx;
  uint8_t* q = Q + static_cast<int64_t>(live ? m : 0) * ldq;
  const int n = live ? K : 0;

  float amax = 0.f;
  constexpr int STEP = VEC ? 8 * T : T;
  constexpr int HELD = VEC ? kCached : 1;
  uint4 c[HELD];
  if constexpr (VEC) {
#pragma unroll
    for (int ch = 0; ch < HELD; ++ch) {
      const int k = ch * STEP + 8 * t;
      c[ch] = make_uint4(0u, 0u, 0u, 0u);
      if (k < n) {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + k));
        c[ch] = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
#pragma unroll
    for (int ch = 0; ch < HELD; ++ch) amax = amax8(amax, c[ch]);
    for (int k = HELD * STEP + 8 * t; k < n; k += STEP)
      amax = amax8(amax, *reinterpret_cast<const uint4*>(x + k));
  } else {
    for (int k = t; k < n; k += STEP) amax = fmaxf(amax, fabsf(bf16_bits_to_f32(x[k])));
  }
  amax = wave_max(amax);
  if constexpr (W > 1) {
    if ((t & 63) == 0) part[t >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) amax = fmaxf(amax, part[w]);
  }
  const float s = amax > 0.f ? amax / 127.f : 1.f;
  if (live && t == 0) scale[m] = s;
  if constexpr (VEC) {
#pragma unroll
    for (int ch = 0; ch < HELD; ++ch) {
      const int k = ch * STEP + 8 * t;
      if (k < n) {
        const uint2 w = int8_codes8(c[ch], s);
        __builtin_nontemporal_store(u32x2{w.x, w.y}, reinterpret_cast<u32x2*>(q + k));
      }
    }
    for (int k = HELD * STEP + 8 * t; k < n; k += STEP)
      *reinterpret_cast<uint2*>(q + k) = int8_codes8(*reinterpret_cast<const uint4*>(x + k), s);
  } else {
    for (int k = t; k < n; k += STEP)
      q[k] = static_cast<uint8_t>(quant_i8(bf16_bits_to_f32(x[k]) / s, 1.f, 0.f));
  }
}

hipError_t launch_quantize_int8_rows(int64_t M, int64_t K, const void* X, int64_t ldx, void* Q,
                                     int64_t ldq, float* scale, bool vec, hipStream_t stream) {
  // Four waves per row where one would not hold it, or where there are too
  // few rows to fill the chip with a wave each (8192 rows of 14336: 65 us,
  // 5.4 TB/s).
  const bool wide = K > kCached * kChunk || M < 1024;
  const int64_t rows_per_wg = wide ? 1 : kQuantThreads / 64;
  const dim3 grid(static_cast<unsigned>((M + rows_per_wg - 1) / rows_per_wg)), block(kQuantThreads);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, static_cast<const uint16_t*>(X), ldx,
                       static_cast<uint8_t*>(Q), ldq, scale, static_cast<int>(M),
                       static_cast<int>(K));
  };
  if (wide) vec ? go(quantize_int8_rows_kernel<4, true>) : go(quantize_int8_rows_kernel<4, false>);
  else vec ? go(quantize_int8_rows_kernel<1, true>) : go(quantize_int8_rows_kernel<1, false>);
  return hipGetLastError();
}

// sums[n] = sum_k b(k, n) of INT8 K-major rows, one wave per row: the weight's
// share of a zero point. Read once when a weight is loaded.
__global__ void __launch_bounds__(kQuantThreads)
int8_row_sums_kernel(const int8_t* __restrict__ B, int64_t ldb, int32_t* __restrict__ sums, int N,
                     int K, bool vec) {
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * (kQuantThreads / 64) + (threadIdx.x >> 6);
  if (n >= N) return;
  const int8_t* b = B + static_cast<int64_t>(n) * ldb;
  int sum = 0, k = lane;
  if (vec) {
    const int whole = K & ~15;
    for (int i = 16 * lane; i < whole; i += 1024) {
      const uint4 v = *reinterpret_cast<const uint4*>(b + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += static_cast<int8_t>(w[j] >> (8 * e));
    }
    k = whole + lane;
  }
  for (; k < K; k += 64) sum += b[k];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) sums[n] = sum;
}

hipError_t launch_int8_row_sums(int64_t N, int64_t K, const void* B, int64_t ldb, int32_t* sums,
                                hipStream_t stream) {
  const int rows_per_wg = kQuantThreads / 64;
  const dim3 grid(static_cast<unsigned>((N + rows_per_wg - 1) / rows_per_wg)), block(kQuantThreads);
  const bool vec = (reinterpret_cast<uintptr_t>(B) & 15u) == 0 && ldb % 16 == 0;
  hipLaunchKernelGGL(int8_row_sums_kernel, grid, block, 0, stream, static_cast<const int8_t*>(B),
                     ldb, sums, static_cast<int>(N), static_cast<int>(K), vec);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(int64_t M, int64_t K, const void* X, int64_t ldx, void* Q,
                                int64_t ldq, float* scale, bool vec, hipStream_t stream) {
  const int rows_per_wg = kQuantThreads / 64;
  const dim3 grid(static_cast<unsigned>((M + rows_per_wg - 1) / rows_per_wg)), block(kQuantThreads);
  if (vec)
    hipLaunchKernelGGL((quantize_rows_kernel<true>), grid, block, 0, stream,
                       static_cast<const uint16_t*>(X), ldx, static_cast<uint8_t*>(Q), ldq, scale,
                       static_cast<int>(M), static_cast<int>(K));
  else
    hipLaunchKernelGGL((quantize_rows_kernel<false>), grid, block, 0, stream,
                       static_cast<const uint16_t*>(X), ldx, static_cast<uint8_t*>(Q), ldq, scale,
                       static_cast<int>(M), static_cast<int>(K));
  return hipGetLastError();
}

}  // namespace g355
