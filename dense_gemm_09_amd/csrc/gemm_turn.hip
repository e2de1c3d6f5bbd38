// 256x256 tiles, two groups of four waves taking turns at the matrix cores.
//
// The kernel of the INT8 product, of the products grouped by rows and of their
// weight gradient wherever an output is large enough for 256x256 tiles. What
// bounds a tile kernel here is feeding the matrix cores: a SIMD holds two waves,
// and one that reads fragments, issues copies and multiplies in a single
// instruction stream leaves the matrix core idle at every wait. So the two
// waves of a SIMD alternate:
//
// * The K slice (128 bytes of every row, two LDS buffers of 64 KB) is worked
//   off in four quarters, each the product of one half of the wave's rows (64)
//   and one half of its columns (32) over the whole slice. A turn reads the
//   fragments that its quarter adds, issues an eighth of the copies of a later
//   slice, then multiplies; barriers on both sides of the multiplications keep
//   waves 0-3 half a turn ahead of waves 4-7, so that on every SIMD one wave
//   multiplies while the other reads. The order A0B0, A0B1, A1B1, A1B0 and, on
//   odd slices, the same with B0 and B1 exchanged, needs 8, 4, 8 and 4 new
//   fragments, and holds one half of A's and both of B's.
// * A half of a buffer whose fragments were read in turn t is refilled from
//   turn t+2 on: at most 2 copies a turn, each with five turns to arrive. Copies
//   complete in order, so a fixed count (vmcnt 10) is all that a turn waits for.
// * 16x16 MFMAs (32 BF16, 64 INT8 or 128 FP8 elements of K). The same loop with
//   the 32x32 shapes of the tile kernel ran 1316 instead of 1191 us (16384 x
//   14336 x 4096, BF16) and 696 instead of 620 us (INT8).
// * C is computed transposed (B's fragment first): a lane then holds 4
//   consecutive columns of one row per MFMA block, and the order of B's rows in
//   a fragment makes that 8 for BF16 outputs. The epilogue works on registers
//   and stores 16 bytes per lane, 64 contiguous bytes per row, without LDS.
//
// Operands that are contiguous along the other axis (the weight of an input
// gradient, both operands of a weight gradient) are copied as they lie: LDS
// then holds 64 rows of K, and fragments come from transposing reads.

#include <type_traits>

#include "common.hpp"
#include "grouping.hpp"
#include "internal.hpp"

namespace g355 {

constexpr int kTurnThreads = 512;
constexpr int kBuf = 32768;     // one operand's slice
constexpr int kHalf = 16384;    // half of its rows (or columns)
constexpr int kBBase = 65536;   // B's two slices follow A's
constexpr int kAhead = 10;      // copies of later turns that may be in flight

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
// Global vectors at any element alignment (the hardware takes them).
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

template <int TY_, int OUT_, bool AR_, bool BR_, int MODE_>
struct TurnCfg {
  static constexpr int TY = TY_, OUT = OUT_, MODE = MODE_;
  static constexpr bool AR = AR_, BR = BR_;  // operand contiguous along its rows' axis, not K
  static constexpr int ES = TY == TY_BF16 ? 2 : 1;
  static constexpr int BKE = 128 / ES;       // K elements per slice
  static constexpr int CE = 16 / ES;         // K elements per 16-byte chunk
  static_assert(TY == TY_BF16 || (!AR && !BR), "rows of one byte: K-major only");
  // BF16 outputs: column 8q + 4u + e of a 32-column half is element e of lane
  // group q of MFMA block u; FP32: column 16u + 4q + e.
  static constexpr bool PAIR = OUT == OUT_BF16;
  using Acc = std::conditional_t<TY == TY_I8, i32x4, f32x4>;
};

// Chunk c of row r of a K-major tile is stored at c ^ swizzle(r). A fragment
// read takes one chunk of 16 rows: consecutive ones (A; B for FP32 outputs), or
// (PAIRED) those that differ in bits 0, 1, 3 and 4. Either way every 8 and
// every 16 consecutive lanes touch distinct 16-byte slots of the 64 banks.
template <bool PAIRED>
__device__ __forceinline__ int turn_swizzle(int r) {
  if constexpr (PAIRED) return ((r >> 3) & 1) | (r & 2) | ((((r >> 4) ^ r) & 1) << 2);
  else return (r & 7) ^ ((r >> 3) & 1);
}

// Chunk c of row k of an operand copied as rows of 128 columns (256 bytes) is
// stored at c ^ rows_swizzle(k): the four rows of a transposing read, whose
// pieces span 32 bytes (or 64, PAIRED), then lie on different banks.
template <bool PAIRED>
__device__ __forceinline__ int rows_swizzle(int k) {
  if constexpr (PAIRED) return 4 * (k & 3);
  else return 2 * (k & 3) + 8 * ((k >> 3) & 1);
}

// ------------------------------------------------------------------------ copies

// K-major operand: each wave copies 16 rows of a half in two instructions of
// eight rows of 128 bytes. Rows past the operand's end repeat its last row
// (their results are never stored); chunks that do not end by k_end read zeros:
// they get an offset past the descriptor's range.
template <class C, bool PAIRED>
struct KMajorCopy {
  uint32_t off[2][2];
  int last[2];  // K element after the lane's chunk, slice-relative
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t extent;
  __device__ __forceinline__ void init(const void* ptr, int64_t ld, int row0, int rows, int K,
                                       int wave, int lane) {
    extent = static_cast<uint32_t>((static_cast<int64_t>(rows - 1) * ld + K) * C::ES);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(ptr), 0, static_cast<int>(extent),
                                             kBufferWord3);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = 16 * wave + 8 * q + (lane >> 3);
      const int c = (lane & 7) ^ turn_swizzle<PAIRED>(r);
      last[q] = c * C::CE + C::CE;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = min(row0 + 128 * h + r, rows - 1);
        off[h][q] = static_cast<uint32_t>(static_cast<int64_t>(g) * ld * C::ES) + c * 16;
      }
    }
  }
  __device__ __forceinline__ void issue(char* half, int h, int wave, int k0, int k_end) const {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t vo = k0 + last[q] <= k_end ? off[h][q] : extent;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (G355_LDS void*)(half + (2 * wave + q) * 1024),
                                               16, static_cast<int>(vo), k0 * C::ES, 0, 0);
    }
  }
};

// Operand whose rows run along K (BF16): a half is 128 of its columns, each
// wave copies eight rows of them. The descriptor's base moves with the slice,
// so that any number of rows can be addressed, and its range ends with row
// k_end - 1, so that later rows read zeros. A chunk that straddles the last
// column brings in what follows the row, for columns that are never stored. The
// range check drops a 4-byte word that lies partly past the range, which for an
// odd column count holds the last element: the range is 2 bytes longer (the
// host makes sure that those stay on the operand's last page).
template <class C, bool PAIRED>
struct RowsCopy {
  uint32_t off[2][2];
  const char* base;
  int64_t ld2;  // bytes per row
  int cols;
  __device__ __forceinline__ void init(const void* ptr, int64_t ld, int col0, int cols_, int,
                                       int wave, int lane) {
    base = static_cast<const char*>(ptr);
    ld2 = ld * 2;
    cols = cols_;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 8 * wave + 4 * q + (lane >> 4);
      const int c = (lane & 15) ^ rows_swizzle<PAIRED>(k);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = col0 + 128 * h + 8 * c;
        off[h][q] = n < cols ? static_cast<uint32_t>(k * ld2 + n * 2) : 0x80000000u;
      }
    }
  }
  __device__ __forceinline__ void issue(char* half, int h, int wave, int k0, int k_end) const {
    const int rem = k_end - k0;
    const int64_t want = rem > 0 ? (rem - 1) * ld2 + cols * 2 + 2 : 0;
    const int range = static_cast<int>(want < INT32_MAX ? want : INT32_MAX);
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base + k0 * ld2), 0, range, kBufferWord3);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (G355_LDS void*)(half + (2 * wave + q) * 1024),
                                               16, static_cast<int>(off[h][q]), 0, 0, 0);
  }
};

// --------------------------------------------------------------------- fragments

// Fragments of one operand: NB blocks of 16 rows (columns of C) per half, two
// 16-byte pieces each (64 bytes of K a piece over the four lane groups).
template <class C, int NB, bool ROWS, bool PAIRED>
struct Fragments {
  // ROWS, not PAIRED: the swizzle reaches the bits that tell blocks apart, so
  // every block has an address of its own.
  static constexpr int NA = ROWS ? (PAIRED ? 1 : NB) : 2;
  int addr[NA];

  // row0: the wave's first row in a half (a multiple of 16 * NB).
  __device__ __forceinline__ void init(int base, int row0, int lane) {
    const int d = lane & 15, g = lane >> 4;
    if constexpr (!ROWS) {
      // Row d of block b: 16 b + d, or PAIRED 8 (d / 4) + 4 b + d % 4.
      const int r = row0 + (PAIRED ? 8 * (d >> 2) + (d & 3) : d);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        addr[t] = base + r * 128 + (((4 * t + g) ^ turn_swizzle<PAIRED>(r)) << 4);
    } else {
      // Lane d of a group points at row d / 4 of four and at 4 columns of it;
      // it receives column d (PAIRED: 8 (d / 4) + 4 b + d % 4) of the four rows.
      const int k = 8 * g + (d >> 2);
#pragma unroll
      for (int b = 0; b < NA; ++b) {
        const int c = PAIRED ? (row0 >> 3) + (d & 3) : ((row0 + 16 * b) >> 3) + ((d & 3) >> 1);
        addr[b] = base + k * 256 + ((c ^ rows_swizzle<PAIRED>(k)) << 4) + (PAIRED ? 0 : 8 * (d & 1));
      }
    }
  }

  // Piece t of block b in the half that starts `at` bytes into the operand's LDS.
  __device__ __forceinline__ i32x4 read(const char* smem, int at, int b, int t) const {
    if constexpr (!ROWS) {
      return *reinterpret_cast<const i32x4*>(smem + addr[t] + at + b * (PAIRED ? 4 : 16) * 128);
    } else {
      const char* q = smem + addr[PAIRED ? 0 : b] + at + t * 32 * 256 + (PAIRED ? 8 * b : 0);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((G355_LDS s16x4*)q);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((G355_LDS s16x4*)(q + 4 * 256));
      return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// acc += the product of two blocks over the 128 bytes of K in pieces 0 and 1.
template <class C>
__device__ __forceinline__ void turn_mfma(typename C::Acc& acc, const i32x4 (&x)[2],
                                          const i32x4 (&y)[2], int t) {
  if constexpr (C::TY == TY_FP8) {
    // One MFMA takes both pieces.
    if (t == 0)
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7),
          __builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7), acc, 0, 0, 0, 127, 0, 127);
  } else if constexpr (C::TY == TY_I8) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[t], y[t], acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[t]),
                                                  __builtin_bit_cast(bf16x8, y[t]), acc, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------- epilogue

// C = act(alpha * scale_a[m] * scale_b[n] * acc + beta * C + bias[n]) from the
// registers. Lane l of block (i, j) holds row 16 i + l % 16 (in its half) and
// the columns of TurnCfg::PAIR. row0, col0: the wave's first row and column.
// ZERO: INT8 with zero points.
template <class C, int ACT, bool ZERO>
__device__ __forceinline__ void turn_epilogue(const GemmArgs& p, const typename C::Acc (&acc)[8][4],
                                              int row0, int col0, int lane) {
  constexpr bool SCALED = C::ES == 1;
  constexpr int W = C::PAIR ? 8 : 4;   // consecutive columns per store
  constexpr int RUNS = 16 / W;
  const int q = lane >> 4, r = lane & 15;
  int n0[RUNS];
#pragma unroll
  for (int s = 0; s < RUNS; ++s)
    n0[s] = col0 + (C::PAIR ? 128 * s + 8 * q : 128 * (s >> 1) + 16 * (s & 1) + 4 * q);

  float cs[16], bias[16];
  int zb[16];
#pragma unroll
  for (int s = 0; s < RUNS; ++s)
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int n = n0[s] + e, x = s * W + e;
      const bool in = n < p.N;
      cs[x] = p.alpha;
      if constexpr (SCALED) cs[x] = in ? p.alpha * p.scale_b[n] : 0.f;
      bias[x] = p.bias && in ? bf16_bits_to_f32(p.bias[n]) : 0.f;
      zb[x] = 0;
      if (ZERO && in) zb[x] = p.sum_b[n];
    }
  float sa[8];
  int za[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = min(row0 + 128 * (i >> 2) + 16 * (i & 3) + r, p.M - 1);
    sa[i] = 1.f;
    za[i] = 0;
    if constexpr (SCALED) sa[i] = p.scale_a[m];
    if (ZERO) za[i] = p.zero_a[m];
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = row0 + 128 * (i >> 2) + 16 * (i & 3) + r;
    if (m >= p.M) continue;
#pragma unroll
    for (int s = 0; s < RUNS; ++s) {
      const int n = n0[s];
      if (n >= p.N) continue;
      const int64_t off = static_cast<int64_t>(m) * p.ldc + n;
      const bool whole = n + W <= p.N;
      float v[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const auto a = acc[i][C::PAIR ? 2 * s + (e >> 2) : s][e & 3];
        float z;
        if constexpr (C::TY == TY_I8) z = i8_sum(a, ZERO, za[i], static_cast<double>(zb[s * W + e]));
        else z = a;
        v[e] = fmaf(z, SCALED ? sa[i] * cs[s * W + e] : cs[s * W + e], bias[s * W + e]);
      }
      if (p.beta != 0.f) {
        float c[W];
        if (whole) {
          if constexpr (C::OUT == OUT_BF16) {
            const u32x4 h = *reinterpret_cast<const u32x4_at2*>(static_cast<const uint16_t*>(p.C) + off);
#pragma unroll
            for (int e = 0; e < W; ++e)
              c[e] = __uint_as_float(e & 1 ? h[e >> 1] & 0xffff0000u : h[e >> 1] << 16);
          } else {
            const f32x4 h = *reinterpret_cast<const f32x4_at4*>(static_cast<const float*>(p.C) + off);
#pragma unroll
            for (int e = 0; e < W; ++e) c[e] = h[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) c[e] = n + e < p.N ? load_cin1<C::OUT>(p.C, off + e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = fmaf(p.beta, c[e], v[e]);
      }
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = apply_act<C::OUT>(v[e], ACT);
      if (whole) {
        if constexpr (C::OUT == OUT_BF16) {
          u32x4 h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = f32x2_to_bf16x2_bits(v[2 * e], v[2 * e + 1]);
          __builtin_nontemporal_store(h, reinterpret_cast<u32x4_at2*>(static_cast<uint16_t*>(p.C) + off));
        } else {
          __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]},
                                      reinterpret_cast<f32x4_at4*>(static_cast<float*>(p.C) + off));
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (n + e < p.N) store_out1<C::OUT>(p.C, off + e, v[e], 1.f, 0.f);
      }
    }
  }
}

// Runs the epilogue with the activation as a compile-time parameter.
template <class C, bool ZERO>
__device__ __forceinline__ void turn_epilogues(const GemmArgs& p, const typename C::Acc (&acc)[8][4],
                                               int row0, int col0, int lane) {
  const int act = p.act;
  if (act == ACT_NONE) turn_epilogue<C, ACT_NONE, ZERO>(p, acc, row0, col0, lane);
  else if (act == ACT_RELU) turn_epilogue<C, ACT_RELU, ZERO>(p, acc, row0, col0, lane);
  else if (act == ACT_GELU_ERF) turn_epilogue<C, ACT_GELU_ERF, ZERO>(p, acc, row0, col0, lane);
  else turn_epilogue<C, ACT_GELU_TANH, ZERO>(p, acc, row0, col0, lane);
}

// ------------------------------------------------------------------------ kernel

// Nothing is moved across a fence, neither by the optimiser nor by the scheduler.
__device__ __forceinline__ void fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void turn_barrier() {
  fence();
  __builtin_amdgcn_s_barrier();
  fence();
}

template <class C>
__global__ void __launch_bounds__(kTurnThreads, 2) gemm_turn_kernel(GemmArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char smem[131072];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  int tm, tn;
  if constexpr (C::MODE == MODE_DENSE) {
    tile_coords(xcd_remap(blockIdx.x, gridDim.x), p.tiles_m, p.tiles_n, 4, tm, tn);
  } else if constexpr (C::MODE == MODE_GROUPED) {
    int L, g, s, rows, tiles, first;
    if (!find_group<256>(p, blockIdx.x, lane, L, g, s, rows, tiles, first)) return;
    tile_coords(L - first * p.tiles_n, tiles, p.tiles_n, kGroupedBand, tm, tn);
    // The operands of this row tile alone, its first row as row 0: 64-bit
    // pointer arithmetic here, so that 32-bit offsets never see more than a
    // tile's rows or one group's weight.
    const int r0 = s + tm * 256;
    p.A = static_cast<const char*>(p.A) + r0 * p.lda * C::ES;
    p.C = static_cast<char*>(p.C) + r0 * p.ldc * (C::OUT == OUT_F32 ? 4 : 2);
    p.M = min(rows - tm * 256, 256);
    tm = 0;
    p.B = static_cast<const char*>(p.B) + g * p.stride_b * C::ES;
    const int64_t gn = static_cast<int64_t>(g) * p.N;
    if (p.bias) p.bias += gn;
    if constexpr (C::ES == 1) {
      p.scale_a += r0;
      p.scale_b += gn;
      if (p.zero_a) {
        p.zero_a += r0;
        p.sum_b += gn;
      }
    }
  } else {
    int g, s, e;
    if (!wgrad_tile(p, blockIdx.x, g, tm, tn)) return;
    group_rows(p, g, s, e);
    p.K = __builtin_amdgcn_readfirstlane(e - s);
    s = __builtin_amdgcn_readfirstlane(s);
    p.A = static_cast<const char*>(p.A) + s * p.lda * C::ES;
    p.B = static_cast<const char*>(p.B) + s * p.ldb * C::ES;
    p.C = static_cast<char*>(p.C) + g * p.stride_b * (C::OUT == OUT_F32 ? 4 : 2);
  }
  const int m0 = tm * 256, n0 = tn * 256, k_end = p.K;
  const int nk = (k_end + C::BKE - 1) / C::BKE;

  std::conditional_t<C::AR, RowsCopy<C, false>, KMajorCopy<C, false>> ca;
  std::conditional_t<C::BR, RowsCopy<C, C::PAIR>, KMajorCopy<C, C::PAIR>> cb;
  ca.init(p.A, p.lda, m0, p.M, p.K, wave, lane);
  cb.init(p.B, p.ldb, n0, p.N, p.K, wave, lane);
  Fragments<C, 4, C::AR, false> ra;
  Fragments<C, 2, C::BR, C::PAIR> rb;
  ra.init(0, 64 * (wave >> 2), lane);
  rb.init(kBBase, 32 * (wave & 3), lane);

  typename C::Acc acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = typename C::Acc{0, 0, 0, 0};
  i32x4 fa[4][2], fb[2][2][2];

  auto copy_a = [&](int buf, int h, int s) __attribute__((always_inline)) {
    ca.issue(smem + buf * kBuf + h * kHalf, h, wave, s * C::BKE, k_end);
  };
  auto copy_b = [&](int buf, int h, int s) __attribute__((always_inline)) {
    cb.issue(smem + kBBase + buf * kBuf + h * kHalf, h, wave, s * C::BKE, k_end);
  };
  auto read_a = [&](int buf, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int b = 0; b < 4; ++b) fa[b][t] = ra.read(smem, buf * kBuf + h * kHalf, b, t);
  };
  auto read_b = [&](int buf, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) fb[h][b][t] = rb.read(smem, buf * kBuf + h * kHalf, b, t);
  };
  // The second half of a turn: the quarter (ha, hb), between two barriers.
  auto multiply = [&](int ha, int hb) __attribute__((always_inline)) {
    fence();
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kAhead) : "memory");
    turn_barrier();
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          turn_mfma<C>(acc[4 * ha + i][2 * hb + j], fb[hb][j], fa[i], t);
    // This turn's reads are done: from the next turn but one their LDS may be refilled.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    turn_barrier();
  };
  // Slice s in buffer f; half f of its B is in registers, and turn 4 reads the
  // half that the next slice starts with.
  auto slice = [&](const int f, int s) __attribute__((always_inline)) {
    read_a(f, 0);
    copy_a(1 - f, 1, s + 1);
    multiply(0, f);
    read_b(f, 1 - f);
    copy_b(f, f, s + 2);
    multiply(0, 1 - f);
    read_a(f, 1);
    copy_a(f, 0, s + 2);
    multiply(1, 1 - f);
    read_b(1 - f, 1 - f);
    copy_b(f, 1 - f, s + 2);
    multiply(1, f);
  };

  if (nk > 0) {
    // The copies that the turns before slice 0 would have issued, in their order.
    copy_b(0, 0, 0);
    copy_a(0, 0, 0);
    copy_b(0, 1, 0);
    copy_a(0, 1, 0);
    copy_b(1, 1, 1);
    copy_a(1, 0, 1);
    copy_b(1, 0, 1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kAhead) : "memory");
    turn_barrier();
    read_b(0, 0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (wave >= 4) turn_barrier();  // half a turn behind waves 0-3
    int s = 0;
    for (; s + 1 < nk; s += 2) {
      slice(0, s);
      slice(1, s + 1);
    }
    if (s < nk) slice(0, s);
    if (wave < 4) turn_barrier();
    // Copies past the end (of zeros) may still be writing LDS.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    turn_barrier();
    // K ends inside a 16-byte chunk of K-major rows: no copy took that chunk,
    // as its bytes past the end may lie past the allocation. One thread per
    // row of A and of B writes it to LDS, zeros after its nb valid bytes, and
    // one more product is added whose other chunks are zero.
    if (!C::AR && k_end % C::CE != 0) {
      const int t = threadIdx.x;
      const bool is_a = t < 256;
      const int tail = k_end % C::CE, nb = tail * C::ES;
      const int row = min((is_a ? m0 : n0) + (t & 255), (is_a ? p.M : p.N) - 1);
      const uintptr_t src = reinterpret_cast<uintptr_t>(is_a ? p.A : p.B) +
                            (row * (is_a ? p.lda : p.ldb) + k_end - tail) * C::ES;
      // Only 4-byte aligned words that hold a valid byte are read.
      const uint32_t* word = reinterpret_cast<const uint32_t*>(src & ~uintptr_t{3});
      const int shift = static_cast<int>(src & 3), words = C::BR && !is_a ? 0 : (shift + nb + 3) >> 2;
      uint32_t d[5], w[4];
#pragma unroll
      for (int i = 0; i < 5; ++i) d[i] = i < words ? word[i] : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = __builtin_amdgcn_alignbyte(d[i + 1], d[i], shift);
        const int keep = nb - 4 * i;
        w[i] = keep >= 4 ? v : keep <= 0 ? 0u : (v & ((1u << (8 * keep)) - 1u));
      }
      if (C::BR && !is_a) {
        // A column of B whose rows run along K: one element of each row.
        const uint16_t* col = static_cast<const uint16_t*>(p.B) + row;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < tail) w[i >> 1] |= static_cast<uint32_t>(col[(k_end - tail + i) * p.ldb]) << (16 * (i & 1));
      }
      *reinterpret_cast<uint4*>(smem + t * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      turn_barrier();
      // Row d of block b of half h as in Fragments.
      const int d16 = lane & 15;
      const auto chunk = [&](int r) {
        i32x4 v = *reinterpret_cast<const i32x4*>(smem + r * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lane < 16 ? v[i] : 0;
        return v;
      };
      const int rowb = 256 + 32 * (wave & 3) + (C::PAIR ? 8 * (d16 >> 2) + (d16 & 3) : d16);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          fb[h][b][0] = chunk(rowb + 128 * h + (C::PAIR ? 4 : 16) * b);
          fb[h][b][1] = i32x4{0, 0, 0, 0};
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const i32x4 x[2] = {chunk(64 * (wave >> 2) + 128 * (i >> 2) + 16 * (i & 3) + d16), i32x4{0, 0, 0, 0}};
#pragma unroll
        for (int j = 0; j < 4; ++j) turn_mfma<C>(acc[i][j], fb[j >> 1][j & 1], x, 0);
      }
    }
  }

  const int row0 = m0 + 64 * (wave >> 2), col0 = n0 + 32 * (wave & 3);
  if constexpr (C::TY == TY_I8) {
    if (p.zero_a) {
      turn_epilogues<C, true>(p, acc, row0, col0, lane);
      return;
    }
  }
  turn_epilogues<C, false>(p, acc, row0, col0, lane);
#endif
}

// --------------------------------------------------------------------- launchers

template <class C>
static hipError_t go(int64_t grid, const GemmArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_turn_kernel<C>), dim3(static_cast<unsigned>(grid)), dim3(kTurnThreads), 0,
                     stream, a);
  return hipGetLastError();
}

// Compiled once per family (G355_TURN), so that they build in parallel.
template <int TY, bool AR, bool BR, int MODE>
static hipError_t by_output(const LaunchSpec& spec, int64_t grid, const GemmArgs& a, hipStream_t s) {
  return spec.out == OUT_F32 ? go<TurnCfg<TY, OUT_F32, AR, BR, MODE>>(grid, a, s)
                             : go<TurnCfg<TY, OUT_BF16, AR, BR, MODE>>(grid, a, s);
}

#if G355_TURN == 0
hipError_t launch_turn_bf16(const LaunchSpec& spec, int64_t grid, const GemmArgs& a, hipStream_t s) {
  return spec.loader_b == LOAD_DIRECT_N ? by_output<TY_BF16, false, true, MODE_GROUPED>(spec, grid, a, s)
                                        : by_output<TY_BF16, false, false, MODE_GROUPED>(spec, grid, a, s);
}
#elif G355_TURN == 1
hipError_t launch_turn_fp8(const LaunchSpec& spec, int64_t grid, const GemmArgs& a, hipStream_t s) {
  return by_output<TY_FP8, false, false, MODE_GROUPED>(spec, grid, a, s);
}
#elif G355_TURN == 2
hipError_t launch_turn_i8(const LaunchSpec& spec, int64_t grid, const GemmArgs& a, hipStream_t s) {
  return a.groups > 0 ? by_output<TY_I8, false, false, MODE_GROUPED>(spec, grid, a, s)
                      : by_output<TY_I8, false, false, MODE_DENSE>(spec, grid, a, s);
}
#else
hipError_t launch_turn_wgrad(const LaunchSpec& spec, int64_t grid, const GemmArgs& a, hipStream_t s) {
  return by_output<TY_BF16, true, true, MODE_WGRAD>(spec, grid, a, s);
}
#endif

}  // namespace g355
