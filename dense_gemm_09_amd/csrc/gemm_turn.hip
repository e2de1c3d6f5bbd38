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
//   the 32x32 shapes of the tile kernel, epilogue left out, ran 1316 instead of
//   1191 us (16384 x 14336 x 4096, BF16) and 696 instead of 620 us (INT8).
// * C is computed transposed (B's fragment first): a lane then holds 4
//   consecutive columns of one row per MFMA block, and the order of B's rows in
//   a fragment makes that 8 for BF16 outputs. The epilogue works on registers
//   and stores 16 bytes per lane, 64 contiguous bytes per row, without LDS. The
//   stores go through the caches, which join the halves of a line: non-temporal
//   ones of this shape reach 2.4-2.8 TB/s, these 5.0 (a fill kernel 6.9).
// * A workgroup per CU takes its tiles as one stream: copies for the next tile
//   are in flight while this one's epilogue runs (8 experts' forward pass, no
//   activation, 1602 -> 1543 us; short products lose nothing).
//
// Measured at 16384 rows over 8 experts, 14336 x 4096, calls over changing inputs,
// one run: forward with bias and GELU 1662 us (1158 TFLOP/s; without them 1572),
// weight gradient in FP32 1780 us. The matrix cores are busy 65% and 55% of the
// cycles and the card runs at its power limit, at 1.6 to 1.8 GHz; GELU is vector
// arithmetic that nothing overlaps (120 us), stores and their acknowledgement cost
// 6 us a tile.
//
// Operands that are contiguous along the other axis (the weight of an input
// gradient, both operands of a weight gradient) are copied as they lie: LDS
// then holds 64 rows of K, and fragments come from transposing reads.

#include <type_traits>

#include "common.hpp"
#include "grouping.hpp"
#include "internal.hpp"
#include "row_copies.hpp"

namespace g355 {

constexpr int kTurnThreads = 512;
constexpr int64_t kTurnGrid = 256;  // a workgroup on every CU
constexpr int kBuf = 32768;     // one operand's slice
constexpr int kHalf = 16384;    // half of its rows (or columns)
constexpr int kBBase = 65536;   // B's two slices follow A's
constexpr int kAhead = 10;      // copies of later turns that may be in flight

typedef int i32x2 __attribute__((ext_vector_type(2)));
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

// Chunk c of row r of a K-major tile is stored at c ^ turn_swizzle(r). A
// fragment read takes chunks c and c ^ 1 of 16 rows in its lanes 0-31 (others in
// 32-63): consecutive rows, or (PAIRED) those that differ in bits 0, 1, 3 and 4.
// The LDS serves lanes 0-3, 12-15 and 20-27 of them at once, then the rest: both
// sets touch 16 distinct 16-byte slots of the 64 banks. (With the tile kernel's
// swizzle, made for 32 rows of one chunk, half of the LDS cycles of these reads
// were conflicts; the counter now reads 0.)
template <bool PAIRED>
__device__ __forceinline__ int turn_swizzle(int r) {
  if constexpr (PAIRED) return ((r >> 1) & 1) | ((r >> 2) & 6);
  else return (r >> 1) & 7;
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
// eight rows of 128 bytes. Rows past the tile's `rows` repeat its last one
// (their results are never stored); chunks that do not end by K read zeros:
// they get an offset past the descriptor's range. Offsets are from the tile's
// first row, 32 bits (the host checks 256 rows).
template <class C, bool PAIRED>
struct KMajorCopy {
  uint32_t off[2][2];
  int last[2];  // K element after the lane's chunk, slice-relative
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t extent;
  __device__ __forceinline__ void next() {}
  __device__ __forceinline__ void point(const char* ptr, int64_t ld, int rows, int K, int wave, int lane) {
    extent = static_cast<uint32_t>((static_cast<uint32_t>(rows - 1) * static_cast<uint32_t>(ld) + K) * C::ES);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(ptr), 0, static_cast<int>(extent),
                                             kBufferWord3);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = 16 * wave + 8 * q + (lane >> 3);
      const int c = (lane & 7) ^ turn_swizzle<PAIRED>(r);
      last[q] = c * C::CE + C::CE;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        off[h][q] = static_cast<uint32_t>(min(128 * h + r, rows - 1)) * static_cast<uint32_t>(ld * C::ES) + c * 16;
    }
  }
  __device__ __forceinline__ void issue(char* half, int h, int wave, int k0, int K) const {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t vo = k0 + last[q] <= K ? off[h][q] : extent;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (G355_LDS void*)(half + (2 * wave + q) * 1024),
                                               16, static_cast<int>(vo), k0 * C::ES, 0, 0);
    }
  }
};

// Operand whose rows run along K (BF16): a half is 128 of its columns, each
// wave copies eight rows of them. The descriptor's base moves with the slice,
// so that any number of rows can be addressed (row_copies.hpp).
template <class C, bool PAIRED>
struct RowsCopy {
  uint32_t off[2][2];
  const char* base;  // of the slice
  int64_t step;      // bytes per slice
  uint32_t ld2;      // bytes per row
  int cols;
  __device__ __forceinline__ void next() { base += step; }
  __device__ __forceinline__ void point(const char* ptr, int64_t ld, int cols_, int K, int wave, int lane) {
    base = ptr;
    static_assert(C::ES == 1 || C::BKE <= kSliceRows, "rows_range");
    ld2 = static_cast<uint32_t>(ld * 2);
    step = ld * 2 * C::BKE;
    cols = cols_;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 8 * wave + 4 * q + (lane >> 4);
      const int c = (lane & 15) ^ rows_swizzle<PAIRED>(k);
#pragma unroll
      for (int h = 0; h < 2; ++h) off[h][q] = rows_offset(k, ld2, 128 * h + 8 * c, cols, K);
    }
  }
  __device__ __forceinline__ void issue(char* half, int h, int wave, int k0, int K) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base), 0, rows_range(K - k0, ld2, cols), kBufferWord3);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (G355_LDS void*)(half + (2 * wave + q) * 1024),
                                               16, static_cast<int>(off[h][q]), 0, 0, 0);
  }
};

// --------------------------------------------------------------------- fragments

// Both pieces of a block's fragment.
__device__ __forceinline__ i32x4 low(const i32x8& x) { return __builtin_shufflevector(x, x, 0, 1, 2, 3); }
__device__ __forceinline__ i32x4 high(const i32x8& x) { return __builtin_shufflevector(x, x, 4, 5, 6, 7); }
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

  // All blocks of the half that starts AT bytes into the operand's LDS.
  template <int AT>
  __device__ __forceinline__ void read(i32x8 (&f)[NB]) const {
    // Written out, with the wait for them: before its own reads of LDS the
    // compiler waits for every copy in flight.
    if constexpr (!ROWS) {
      i32x4 v[NB][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          v[b][t] = *reinterpret_cast<G355_LDS const i32x4*>(addr[t] + AT + b * (PAIRED ? 4 : 16) * 128);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        f[b] = __builtin_shufflevector(v[b][0], v[b][1], 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      i32x2 v[NB][4];
      constexpr int P = PAIRED ? 8 : 0;  // bytes from one block to the next
      if constexpr (NB == 2) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8 offset:%10\n\tds_read_b64_tr_b16 %1, %8 offset:%11\n\t"
            "ds_read_b64_tr_b16 %4, %9 offset:%14\n\tds_read_b64_tr_b16 %5, %9 offset:%15\n\t"
            "ds_read_b64_tr_b16 %2, %8 offset:%12\n\tds_read_b64_tr_b16 %3, %8 offset:%13\n\t"
            "ds_read_b64_tr_b16 %6, %9 offset:%16\n\tds_read_b64_tr_b16 %7, %9 offset:%17\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][2]), "=&v"(v[0][3]), "=&v"(v[1][0]),
              "=&v"(v[1][1]), "=&v"(v[1][2]), "=&v"(v[1][3])
            : "v"(addr[0]), "v"(addr[NA - 1]), "n"(AT), "n"(AT + 1024), "n"(AT + 8192), "n"(AT + 9216),
              "n"(AT + P), "n"(AT + P + 1024), "n"(AT + P + 8192), "n"(AT + P + 9216)
            : "memory");
      } else {
        static_assert(NB == 4 && !PAIRED, "A's blocks");
        asm volatile(
            "ds_read_b64_tr_b16 %0, %16 offset:%20\n\tds_read_b64_tr_b16 %1, %16 offset:%21\n\t"
            "ds_read_b64_tr_b16 %4, %17 offset:%20\n\tds_read_b64_tr_b16 %5, %17 offset:%21\n\t"
            "ds_read_b64_tr_b16 %8, %18 offset:%20\n\tds_read_b64_tr_b16 %9, %18 offset:%21\n\t"
            "ds_read_b64_tr_b16 %12, %19 offset:%20\n\tds_read_b64_tr_b16 %13, %19 offset:%21\n\t"
            "ds_read_b64_tr_b16 %2, %16 offset:%22\n\tds_read_b64_tr_b16 %3, %16 offset:%23\n\t"
            "ds_read_b64_tr_b16 %6, %17 offset:%22\n\tds_read_b64_tr_b16 %7, %17 offset:%23\n\t"
            "ds_read_b64_tr_b16 %10, %18 offset:%22\n\tds_read_b64_tr_b16 %11, %18 offset:%23\n\t"
            "ds_read_b64_tr_b16 %14, %19 offset:%22\n\tds_read_b64_tr_b16 %15, %19 offset:%23\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][2]), "=&v"(v[0][3]), "=&v"(v[1][0]),
              "=&v"(v[1][1]), "=&v"(v[1][2]), "=&v"(v[1][3]), "=&v"(v[2][0]), "=&v"(v[2][1]),
              "=&v"(v[2][2]), "=&v"(v[2][3]), "=&v"(v[3][0]), "=&v"(v[3][1]), "=&v"(v[3][2]),
              "=&v"(v[3][3])
            : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[NA - 1]), "n"(AT), "n"(AT + 1024),
              "n"(AT + 8192), "n"(AT + 9216)
            : "memory");
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
        f[b] = i32x8{v[b][0][0], v[b][0][1], v[b][1][0], v[b][1][1], v[b][2][0], v[b][2][1], v[b][3][0], v[b][3][1]};
    }
  }
};

// acc += the product of two blocks over the 64 bytes of K in piece t (FP8: one
// MFMA takes both pieces, with t = 0).
template <class C>
__device__ __forceinline__ void turn_mfma(typename C::Acc& acc, const i32x8& x, const i32x8& y, int t) {
  if constexpr (C::TY == TY_FP8) {
    if (t == 0)
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, 127, 0, 127);
  } else {
    const i32x4 a = t == 0 ? low(x) : high(x), b = t == 0 ? low(y) : high(y);
    if constexpr (C::TY == TY_I8)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc, 0, 0, 0);
    else
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                    __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------- epilogue

// What a tile's epilogue needs of its rows and columns, in LDS.
struct TileVectors {
  float scale_a[256], scale_b[256];
  int zero_a[256], sum_b[256];
  float bias[256];
};

// C = act(alpha * scale_a[m] * scale_b[n] * acc + beta * C + bias[n]) from the
// registers. Lane l of block (i, j) holds row 16 i + l % 16 (in its half) and
// the columns of TurnCfg::PAIR. c: the tile's first element; row0, col0: the
// wave's first row and column in it. WHOLE: every column exists. ACT: the
// activation, or -1: p.act.
template <class C, int ACT, bool ZERO, bool WHOLE>
__device__ __forceinline__ void turn_epilogue(const GemmArgs& p, const typename C::Acc (&acc)[8][4],
                                              const TileVectors& tv, char* c, int rows, int cols,
                                              int row0, int col0, int lane) {
  constexpr bool SCALED = C::ES == 1;
  constexpr int W = C::PAIR ? 8 : 4;   // consecutive columns per store
  constexpr int RUNS = 8 / W;          // of a half
  constexpr int OB = C::OUT == OUT_F32 ? 4 : 2;
  const int q = lane >> 4, r = lane & 15;
  // Half by half, rows inside: the columns' vectors of one half are in registers.
  // A row's two runs of FP32 fill a 128-byte line one after the other (13
  // gradients of 3200 x 11136: 548 us with the rows between them, 378 so).
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n0 = col0 + 128 * h + W * q;  // run s: n0 + 16 s
    float cs[8], bias[8];
    int zb[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int n = n0 + 16 * (x / W) + x % W;
      cs[x] = p.alpha;
      if constexpr (SCALED) cs[x] = p.alpha * tv.scale_b[n];
      bias[x] = C::MODE != MODE_WGRAD && p.bias ? tv.bias[n] : 0.f;
      zb[x] = 0;
      if (ZERO) zb[x] = tv.sum_b[n];
    }
#pragma unroll
    for (int is = 0; is < 8 * RUNS; ++is) {
      const int i = is / RUNS, s = is % RUNS;
      __builtin_amdgcn_sched_barrier(0);  // one run's registers at a time
      const int n = n0 + 16 * s;
      const int m = row0 + 128 * (i >> 2) + 16 * (i & 3) + r;
      if (m >= rows || (!WHOLE && n >= cols)) continue;
      const bool vec = WHOLE || n + W <= cols;
      float sa = 1.f;
      int za = 0;
      if constexpr (SCALED) sa = tv.scale_a[m];
      if (ZERO) za = tv.zero_a[m];
      char* at = c + m * p.ldc * OB + n * OB;
      float v[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const auto a = acc[i][2 * h + (C::PAIR ? e >> 2 : s)][e & 3];
        float z;
        if constexpr (C::TY == TY_I8) z = i8_sum(a, ZERO, za, static_cast<double>(zb[W * s + e]));
        else z = a;
        v[e] = fmaf(z, SCALED ? sa * cs[W * s + e] : cs[W * s + e], bias[W * s + e]);
      }
      if (p.beta != 0.f) {
        float in[W];
        if (vec) {
          if constexpr (C::OUT == OUT_BF16) {
            const u32x4 h = *reinterpret_cast<const u32x4_at2*>(at);
#pragma unroll
            for (int e = 0; e < W; ++e)
              in[e] = __uint_as_float(e & 1 ? h[e >> 1] & 0xffff0000u : h[e >> 1] << 16);
          } else {
            const f32x4 h = *reinterpret_cast<const f32x4_at4*>(at);
#pragma unroll
            for (int e = 0; e < W; ++e) in[e] = h[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) in[e] = n + e < cols ? load_cin1<C::OUT>(at, e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = fmaf(p.beta, in[e], v[e]);
      }
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = apply_act<C::OUT>(v[e], ACT < 0 ? p.act : ACT);
      if (vec) {
        if constexpr (C::OUT == OUT_BF16) {
          u32x4 h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = f32x2_to_bf16x2_bits(v[2 * e], v[2 * e + 1]);
          *reinterpret_cast<u32x4_at2*>(at) = h;
        } else {
          *reinterpret_cast<f32x4_at4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (n + e < cols) store_out1<C::OUT>(at, e, v[e], 1.f, 0.f);
      }
    }
  }
}

// Runs the epilogue with the activation as a compile-time parameter where
// every column exists.
template <class C, bool ZERO, class... Rest>
__device__ __forceinline__ void turn_epilogues(const GemmArgs& p, const typename C::Acc (&acc)[8][4],
                                               bool whole, const Rest&... rest) {
  if (!whole) {
    turn_epilogue<C, C::MODE == MODE_WGRAD ? static_cast<int>(ACT_NONE) : -1, ZERO, false>(p, acc, rest...);
  } else if constexpr (C::MODE == MODE_WGRAD) {
    turn_epilogue<C, ACT_NONE, ZERO, true>(p, acc, rest...);
  } else {
    const int act = p.act;
    if (act == ACT_NONE) turn_epilogue<C, ACT_NONE, ZERO, true>(p, acc, rest...);
    else if (act == ACT_RELU) turn_epilogue<C, ACT_RELU, ZERO, true>(p, acc, rest...);
    else if (act == ACT_GELU_ERF) turn_epilogue<C, ACT_GELU_ERF, ZERO, true>(p, acc, rest...);
    else turn_epilogue<C, ACT_GELU_TANH, ZERO, true>(p, acc, rest...);
  }
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

// One tile's work: its operands from its first row and column on.
struct TurnTile {
  const char* A;
  const char* B;
  char* C;
  int rows, cols, K;
  int slices;             // even: a last slice past K adds zeros
  int64_t row, col;       // first row of scale_a / zero_a, first element of scale_b, bias, sum_b
};

// Everything a workgroup keeps in LDS: the operands' slices (A's, then B's),
// the vectors of two tiles (the one whose copies run and the one before), the
// groups' tiles, and the last chunks of a K that ends inside one.
struct TurnShared {
  char ring[131072];
  TileVectors vectors[2];
  GroupTable groups;
  uint4 tail[512];
};
static_assert(sizeof(TurnShared) <= 160 * 1024, "LDS budget");

// A pointer that is the same in every lane, in scalar registers (a descriptor
// made of one in vector registers would cost a loop at every copy).
template <class T>
__device__ __forceinline__ T* scalar(T* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  return reinterpret_cast<T*>(lo | static_cast<uint64_t>(hi) << 32);
}

// The workgroup's tile number `v`, or its next one if there is none of that number (false: no more).
template <class C>
__device__ __forceinline__ bool turn_tile(const GemmArgs& p, const TurnShared& sh, int nwg, int& v, int lane,
                                          TurnTile& t) {
  if (v >= nwg) return false;
  constexpr int OB = C::OUT == OUT_F32 ? 4 : 2;
  int tm, tn, rows = p.M, K = p.K;
  int64_t r0 = 0;  // first row of the group
  const char* A = static_cast<const char*>(p.A);
  const char* B = static_cast<const char*>(p.B);
  char* c = static_cast<char*>(p.C);
  t.col = 0;
  if constexpr (C::MODE == MODE_DENSE) {
    tile_coords(xcd_remap(v, nwg), p.tiles_m, p.tiles_n, 4, tm, tn);
  } else if constexpr (C::MODE == MODE_GROUPED) {
    const int L = xcd_remap(v, nwg);
    int g, s, tiles, first;
    find_in_table(sh.groups, L / p.tiles_n, p.groups, lane, g, s, rows, tiles, first);
    tile_coords(L - first * p.tiles_n, tiles, p.tiles_n, kGroupedBand, tm, tn);
    r0 = s;
    B += g * p.stride_b * C::ES;
    t.col = static_cast<int64_t>(g) * p.N;
  } else {
    int g, s, e;
    while (!wgrad_tile(p, v, g, tm, tn))
      if ((v += gridDim.x) >= nwg) return false;
    group_rows(p, g, s, e);
    s = __builtin_amdgcn_readfirstlane(s);
    K = __builtin_amdgcn_readfirstlane(e) - s;
    A += s * p.lda * C::ES;
    B += s * p.ldb * C::ES;
    c += g * p.stride_b * OB;
  }
  const int m0 = tm * 256, n0 = tn * 256;
  t.rows = min(rows - m0, 256);
  t.cols = min(p.N - n0, 256);
  t.row = r0 + m0;
  t.col += n0;
  t.A = scalar(A + t.row * (C::AR ? 1 : p.lda) * C::ES);
  t.B = scalar(B + n0 * (C::BR ? 1 : p.ldb) * C::ES);
  t.C = scalar(c + (t.row * p.ldc + n0) * OB);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.cols = __builtin_amdgcn_readfirstlane(t.cols);
  t.K = __builtin_amdgcn_readfirstlane(K);
  t.slices = 2 * max(1, (t.K + 2 * C::BKE - 1) / (2 * C::BKE));
  return true;
}

// The same value through a move that the optimiser cannot look through: what
// is computed from it stays where it is used, instead of being hoisted out of
// the loop over tiles, where it would hold a register throughout.
__device__ __forceinline__ int opaque(int x) {
  int y;
  asm volatile("v_mov_b32 %0, %1" : "=v"(y) : "v"(x));
  return y;
}

template <class C>
__global__ void __launch_bounds__(kTurnThreads, 2) gemm_turn_kernel(GemmArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) TurnShared sh;
  char* const smem = sh.ring;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // A workgroup takes tiles v, v + gridDim.x, ... as one stream of slices: the
  // copies run ahead into the next tile, so that neither a tile's start nor
  // its stores leave the matrix cores without operands.
  int v = blockIdx.x, nwg = p.turn_tiles;
  if constexpr (C::MODE == MODE_GROUPED) {
    fill_table<256>(p, sh.groups, wave, lane);
    __syncthreads();
    nwg = __builtin_amdgcn_readfirstlane(sh.groups.row_tiles) * p.tiles_n;
  }
  TurnTile cur, nxt;
  bool more = turn_tile<C>(p, sh, nwg, v, lane, cur);
  if (!more) return;

  std::conditional_t<C::AR, RowsCopy<C, false>, KMajorCopy<C, false>> ca;
  std::conditional_t<C::BR, RowsCopy<C, C::PAIR>, KMajorCopy<C, C::PAIR>> cb;
  Fragments<C, 4, C::AR, false> ra;
  Fragments<C, 2, C::BR, C::PAIR> rb;

  // The copies' place in the stream: K0 of their slice, and what is left of their tile.
  int ck0 = 0, cK = 0, cleft = 0;
  const auto point = [&](const TurnTile& t) __attribute__((always_inline)) {
    const int l = opaque(lane);
    ca.point(t.A, p.lda, t.rows, t.K, wave, l);
    cb.point(t.B, p.ldb, t.cols, t.K, wave, l);
    ck0 = 0;
    cK = t.K;
    cleft = t.slices;
  };
  // A tile's vectors pass through three registers of a thread (the first 256
  // threads: its rows' and the bias, the others: its columns').
  constexpr bool VECTORS = C::MODE != MODE_WGRAD;
  float vec0 = 0.f, vec2 = 0.f;
  int vec1 = 0;
  const auto load_vectors = [&](const TurnTile& t) __attribute__((always_inline)) {
    const int id = opaque(tid);
    const bool of_a = id < 256;
    const int x = id & 255;
    if constexpr (C::ES == 1) {
      const bool in = x < (of_a ? t.rows : t.cols);
      if (in) vec0 = of_a ? p.scale_a[t.row + x] : p.scale_b[t.col + x];
      if constexpr (C::TY == TY_I8) {
        if (p.zero_a && in) vec1 = of_a ? p.zero_a[t.row + x] : p.sum_b[t.col + x];
      }
    }
    if (p.bias && of_a && x < t.cols) vec2 = bf16_bits_to_f32(p.bias[t.col + x]);
  };
  const auto store_vectors = [&](TileVectors& tv) __attribute__((always_inline)) {
    const int id = opaque(tid), x = id & 255;
    if constexpr (C::ES == 1) {
      (id < 256 ? tv.scale_a : tv.scale_b)[x] = vec0;
      if constexpr (C::TY == TY_I8) (id < 256 ? tv.zero_a : tv.sum_b)[x] = vec1;
    }
    if (id < 256) tv.bias[x] = vec2;
  };

  typename C::Acc acc[8][4];
  i32x8 fa[4], fb[2][2];
  const auto copy_a = [&](int buf, int h) __attribute__((always_inline)) {
    ca.issue(smem + buf * kBuf + h * kHalf, h, wave, ck0, cK);
  };
  const auto copy_b = [&](int buf, int h) __attribute__((always_inline)) {
    // Rows of B that the chunk of A in which K ends belongs to come in the extra
    // product below: here that chunk is zero, and an infinity or NaN may not meet it.
    const int end = C::BR && !C::AR ? cK & ~(C::CE - 1) : cK;
    cb.issue(smem + kBBase + buf * kBuf + h * kHalf, h, wave, ck0, end);
  };
  const auto read_a = [&](auto buf, auto h) __attribute__((always_inline)) {
    ra.template read<decltype(buf)::value * kBuf + decltype(h)::value * kHalf>(fa);
  };
  const auto read_b = [&](auto buf, auto h) __attribute__((always_inline)) {
    constexpr int H = decltype(h)::value;
    rb.template read<decltype(buf)::value * kBuf + H * kHalf>(fb[H]);
  };
  // The second half of a turn: the quarter (ha, hb), between two barriers.
  const auto multiply = [&](int ha, int hb) __attribute__((always_inline)) {
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
    // (Keeps the products on this side of the barrier: they touch no memory.)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(acc[4 * ha + i][2 * hb + j]));
    // This turn's reads are done: from the next turn but one their LDS may be refilled.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    turn_barrier();
  };
  int parity = 0;  // of the tile whose copies run
  bool moved = false;
  // A slice in buffer f; half f of its B is in registers, and turn 4 reads the
  // half that the next slice starts with. A tile has an even number of slices,
  // so the copies pass from one tile to the next in slices of buffer 0.
  using Zero = std::integral_constant<int, 0>;
  using One = std::integral_constant<int, 1>;
  const auto advance = [&]() __attribute__((always_inline)) {
    ck0 += C::BKE;
    --cleft;
    ca.next();
    cb.next();
  };
  const auto slice = [&](auto F) __attribute__((always_inline)) {
    constexpr int f = decltype(F)::value;
    const std::integral_constant<int, 1 - f> G{};
    copy_a(1 - f, 1);
    read_a(F, Zero{});
    advance();
    if (f == 0) {
      moved = cleft == 0;
      if (moved) {
        v += gridDim.x;
        more = turn_tile<C>(p, sh, nwg, v, opaque(lane), nxt);
        if (!more) {
          nxt = cur;
          nxt.K = 0;  // copies of zeros
          nxt.slices = 1 << 30;
        }
        point(nxt);
        if (VECTORS && more) load_vectors(nxt);
      }
    }
    multiply(0, f);
    copy_b(f, f);
    read_b(F, G);
    if (VECTORS && f == 1 && moved) {
      parity ^= 1;
      store_vectors(sh.vectors[parity]);
    }
    multiply(0, 1 - f);
    copy_a(f, 0);
    read_a(F, One{});
    multiply(1, 1 - f);
    copy_b(f, 1 - f);
    read_b(G, G);
    multiply(1, f);
  };

  // The copies that the turns before slice 0 would have issued, in their order.
  point(cur);
  if (VECTORS) {
    load_vectors(cur);
    store_vectors(sh.vectors[0]);
  }
  copy_b(0, 0);
  copy_a(0, 0);
  copy_b(0, 1);
  copy_a(0, 1);
  advance();
  copy_b(1, 1);
  copy_a(1, 0);
  copy_b(1, 0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead) : "memory");
  turn_barrier();
  if (wave >= 4) turn_barrier();  // half a turn behind waves 0-3

  for (;;) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = typename C::Acc{0, 0, 0, 0};
    // (Addresses of fragments are not held over an epilogue either.)
    const int lds = static_cast<int>(reinterpret_cast<uintptr_t>((G355_LDS char*)smem));
    ra.init(lds, 64 * (wave >> 2), opaque(lane));
    rb.init(lds + kBBase, 32 * (wave & 3), opaque(lane));
    // Half 0 of B, read again so that no register holds it over an epilogue.
    read_b(Zero{}, Zero{});
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    for (int s = 0; s < cur.slices; s += 2) {
      slice(Zero{});
      slice(One{});
    }
    // K ends inside a 16-byte chunk of K-major rows: no copy took that chunk,
    // as its bytes past the end may lie past the allocation. One thread per
    // row of A and of B writes it to LDS, zeros after its nb valid bytes, and
    // one more product is added whose other chunks are zero.
    const int tail = C::AR ? 0 : cur.K % C::CE;
    if (tail != 0) {
      const int id = opaque(tid);
      const bool is_a = id < 256;
      const int nb = tail * C::ES;
      const int row = min(id & 255, (is_a ? cur.rows : cur.cols) - 1);
      const uintptr_t src = reinterpret_cast<uintptr_t>(is_a ? cur.A : cur.B) +
                            (row * (is_a ? p.lda : p.ldb) + cur.K - tail) * C::ES;
      // Only 4-byte aligned words that hold a valid byte are read.
      const uint32_t* word = reinterpret_cast<const uint32_t*>(src & ~uintptr_t{3});
      const int shift = static_cast<int>(src & 3), words = C::BR && !is_a ? 0 : (shift + nb + 3) >> 2;
      uint32_t d[5], w[4];
#pragma unroll
      for (int i = 0; i < 5; ++i) d[i] = i < words ? word[i] : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = __builtin_amdgcn_alignbyte(d[i + 1], d[i], shift);
        const int keep = nb - 4 * i;
        w[i] = keep >= 4 ? x : keep <= 0 ? 0u : (x & ((1u << (8 * keep)) - 1u));
      }
      if (C::BR && !is_a) {
        // A column of B whose rows run along K: one element of each row.
        const uint16_t* col = reinterpret_cast<const uint16_t*>(cur.B) + row;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < tail) w[i >> 1] |= static_cast<uint32_t>(col[(cur.K - tail + i) * p.ldb]) << (16 * (i & 1));
      }
      sh.tail[id] = make_uint4(w[0], w[1], w[2], w[3]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      turn_barrier();  // two: waves 4-7 are one barrier behind
      turn_barrier();
      // Row d of block b of half h as in Fragments.
      const int l = id & 63, d16 = l & 15;
      const auto chunk = [&](int r) {
        i32x4 x = *reinterpret_cast<const i32x4*>(&sh.tail[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = l < 16 ? x[i] : 0;
        return __builtin_shufflevector(x, i32x4{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
      };
      const int rowb = 256 + 32 * (wave & 3) + (C::PAIR ? 8 * (d16 >> 2) + (d16 & 3) : d16);
      // (The fragments in registers belong to the next tile.)
      i32x8 y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = chunk(rowb + 128 * (j >> 1) + (C::PAIR ? 4 : 16) * (j & 1));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const i32x8 x = chunk(64 * (wave >> 2) + 128 * (i >> 2) + 16 * (i & 3) + d16);
#pragma unroll
        for (int j = 0; j < 4; ++j) turn_mfma<C>(acc[i][j], y[j], x, 0);
      }
    }

    const bool whole = cur.cols == 256;
    const TileVectors& tv = sh.vectors[parity ^ 1];
    const int row0 = 64 * (wave >> 2), col0 = 32 * (wave & 3), l = opaque(lane);
    bool zero = false;
    if constexpr (C::TY == TY_I8) zero = p.zero_a != nullptr;
    if (zero) turn_epilogues<C, C::TY == TY_I8>(p, acc, whole, tv, cur.C, cur.rows, cur.cols, row0, col0, l);
    else turn_epilogues<C, false>(p, acc, whole, tv, cur.C, cur.rows, cur.cols, row0, col0, l);
    fence();
    if (!more) break;
    cur = nxt;
  }
  if (wave < 4) turn_barrier();
  // Copies of zeros may still be on their way into LDS.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#endif
}

// --------------------------------------------------------------------- launchers

template <class C>
static hipError_t go(int64_t grid, const GemmArgs& a, hipStream_t stream) {
  GemmArgs t = a;
  t.turn_tiles = static_cast<int>(grid);
  hipLaunchKernelGGL((gemm_turn_kernel<C>), dim3(static_cast<unsigned>(grid < kTurnGrid ? grid : kTurnGrid)),
                     dim3(kTurnThreads), 0, stream, t);
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
