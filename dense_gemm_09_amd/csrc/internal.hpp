// Host-side interface between the C ABI layer and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.hpp"

namespace g355 {

// How an operand's K slices reach LDS.
enum Loader : int {
  LOAD_DIRECT = 0,   // K-major, 16-byte aligned rows: global -> LDS DMA, no registers
  LOAD_GENERIC = 1,  // any layout / alignment: element loads through registers
  LOAD_DIRECT_N = 2, // B only, BF16 N-contiguous (row-major): DMA into an N-major LDS tile, fragments by
                     // transposing LDS reads. Dense products: 16-byte aligned rows, N % 8 == 0; grouped
                     // ones: any N and any 2-byte alignment
  LOAD_ROWS = 3,     // both operands of the weight gradient: the same, an operand of any size
};

enum KernelKind : int { KERNEL_TILE = 0, KERNEL_SKINNY = 1 };

struct Plan {
  int kernel;        // KernelKind
  int bm, bn, bk;    // tile (bk in elements)
  int waves;         // waves per workgroup
  int split;         // K partitions
  int k_split_len;   // K elements per partition
  int64_t grid;      // workgroups of the main kernel
  size_t workspace;  // bytes
};

// Chooses the kernel, tile and split for a shape (host arithmetic only).
Plan make_plan(int64_t M, int64_t N, int64_t K, bool fp8);
// The same among the tile kernels alone.
Plan make_tile_plan(int64_t M, int64_t N, int64_t K, bool fp8);

// Largest K of an INT8 product: K * 128 * 128 stays inside INT32.
constexpr int64_t kMaxInt8K = 131071;

// Largest K split a plan uses (the reduction kernel holds that many partials
// per thread).
constexpr int kMaxSplit = 16;

struct LaunchSpec {
  bool fp8;
  int loader_a, loader_b;  // Loader
  bool a_kmajor, b_kmajor; // layout of each operand (true = K contiguous)
  int out;                 // OutKind
  bool mx;                 // FP8 with E8M0 block scales (GemmArgs::mx_a / mx_b)
  bool i8;                 // INT8 operands (fp8 false)
  bool ragged;             // K not a multiple of the 16-byte chunk, a K-major operand DMA-fed
};

// The tile kernels are instantiated per output part, each in a compile of
// its own (gemm_tile.hip built with G355_PART and G355_RAGGED).
enum OutPart : int { PART_SPLIT = 0, PART_F32 = 1, PART_BF16 = 2, PART_I8 = 3, PART_E4M3 = 4 };
constexpr int kOutParts = 5;

#define G355_PART_LAUNCHER_(r, p) launch_tile_r##r##_p##p
#define G355_PART_LAUNCHER(r, p) G355_PART_LAUNCHER_(r, p)
#define G355_DECLARE_PART(r, p)                                                              \
  hipError_t G355_PART_LAUNCHER(r, p)(const Plan& plan, const LaunchSpec& spec,              \
                                      const GemmArgs& args, hipStream_t stream);
G355_DECLARE_PART(0, 0) G355_DECLARE_PART(0, 1) G355_DECLARE_PART(0, 2) G355_DECLARE_PART(0, 3)
G355_DECLARE_PART(0, 4) G355_DECLARE_PART(1, 0) G355_DECLARE_PART(1, 1) G355_DECLARE_PART(1, 2)
G355_DECLARE_PART(1, 3) G355_DECLARE_PART(1, 4)
#undef G355_DECLARE_PART

// INT8 kernels, the same parts.
#define G355_I8_LAUNCHER_(r, p) launch_i8_r##r##_p##p
#define G355_I8_LAUNCHER(r, p) G355_I8_LAUNCHER_(r, p)
#define G355_DECLARE_I8(r, p)                                                                \
  hipError_t G355_I8_LAUNCHER(r, p)(const Plan& plan, const LaunchSpec& spec,                \
                                    const GemmArgs& args, hipStream_t stream);
G355_DECLARE_I8(0, 0) G355_DECLARE_I8(0, 1) G355_DECLARE_I8(0, 2) G355_DECLARE_I8(0, 3)
G355_DECLARE_I8(0, 4) G355_DECLARE_I8(1, 0) G355_DECLARE_I8(1, 1) G355_DECLARE_I8(1, 2)
G355_DECLARE_I8(1, 3) G355_DECLARE_I8(1, 4)
#undef G355_DECLARE_I8

// Products grouped by rows and their weight gradient: FP32 and BF16 output.
struct GroupedPlan;  // grouped_plan.hpp
#define G355_GROUPED_LAUNCHER_(r, p) launch_grouped_r##r##_p##p
#define G355_GROUPED_LAUNCHER(r, p) G355_GROUPED_LAUNCHER_(r, p)
#define G355_WGRAD_LAUNCHER_(p) launch_wgrad_p##p
#define G355_WGRAD_LAUNCHER(p) G355_WGRAD_LAUNCHER_(p)
#define G355_DECLARE_GROUPED(name)                                                           \
  hipError_t name(const GroupedPlan& plan, const LaunchSpec& spec, const GemmArgs& args,     \
                  hipStream_t stream);
G355_DECLARE_GROUPED(G355_GROUPED_LAUNCHER(0, 1)) G355_DECLARE_GROUPED(G355_GROUPED_LAUNCHER(0, 2))
G355_DECLARE_GROUPED(G355_GROUPED_LAUNCHER(1, 1)) G355_DECLARE_GROUPED(G355_GROUPED_LAUNCHER(1, 2))
G355_DECLARE_GROUPED(G355_WGRAD_LAUNCHER(1)) G355_DECLARE_GROUPED(G355_WGRAD_LAUNCHER(2))
#undef G355_DECLARE_GROUPED

// The projection with low-rank adapters: BF16 operands by DMA, FP32 and BF16
// output and split-K partials.
struct LoraArgs;  // lora.hpp
#define G355_LORA_LAUNCHER_(r, p) launch_lora_r##r##_p##p
#define G355_LORA_LAUNCHER(r, p) G355_LORA_LAUNCHER_(r, p)
#define G355_DECLARE_LORA(r, p)                                                              \
  hipError_t G355_LORA_LAUNCHER(r, p)(const Plan& plan, const LoraArgs& args, hipStream_t stream);
G355_DECLARE_LORA(0, 0) G355_DECLARE_LORA(0, 1) G355_DECLARE_LORA(0, 2)
G355_DECLARE_LORA(1, 0) G355_DECLARE_LORA(1, 1) G355_DECLARE_LORA(1, 2)
#undef G355_DECLARE_LORA

// 256x256 tiles with FP32 or BF16 output (gemm_turn.hip), one element type
// each: grouped products (INT8: the dense one too, where groups is 0) and the
// weight gradient.
hipError_t launch_turn_bf16(const LaunchSpec& spec, int64_t grid, const GemmArgs& args, hipStream_t stream);
hipError_t launch_turn_fp8(const LaunchSpec& spec, int64_t grid, const GemmArgs& args, hipStream_t stream);
hipError_t launch_turn_i8(const LaunchSpec& spec, int64_t grid, const GemmArgs& args, hipStream_t stream);
hipError_t launch_turn_wgrad(const LaunchSpec& spec, int64_t grid, const GemmArgs& args, hipStream_t stream);

// Enqueue the tile kernel of a plan (the part launcher for its output kind
// and ragged flag). Returns the HIP error of the launch.
hipError_t launch_tile(const Plan& plan, const LaunchSpec& spec, const GemmArgs& args,
                       hipStream_t stream);
hipError_t launch_skinny(const Plan& plan, const LaunchSpec& spec, const GemmArgs& args,
                         hipStream_t stream);
// The skinny kernel's streaming variant covers K up to 16 waves x 4096/16
// elements; its grid is one workgroup per CU at most.
inline bool skinny_streams(int64_t K) { return K <= 4096; }
// With adapters it holds one fragment of their ranks (32 of the padded ones) too.
inline bool skinny_streams_lora(int64_t K, int64_t pad) { return skinny_streams(K) && pad <= 32; }
inline int64_t skinny_stream_grid(int64_t N) {
  const int64_t blocks = (N + 15) / 16;
  return blocks < 256 ? blocks : 256;
}
hipError_t launch_splitk_reduce(const Plan& plan, const LaunchSpec& spec, const GemmArgs& args,
                                hipStream_t stream);

// Per-token FP8 quantisation of BF16 rows (quant.hip). vec: 16-byte aligned
// rows with K and ldx multiples of 8 and Q rows 8-byte aligned.
hipError_t launch_quantize_rows(int64_t M, int64_t K, const void* X, int64_t ldx, void* Q,
                                int64_t ldq, float* scale, bool vec, hipStream_t stream);

// The same for INT8 codes, and the row sums of an INT8 weight (quant.hip).
hipError_t launch_quantize_int8_rows(int64_t M, int64_t K, const void* X, int64_t ldx, void* Q,
                                     int64_t ldq, float* scale, bool vec, hipStream_t stream);
hipError_t launch_int8_row_sums(int64_t N, int64_t K, const void* B, int64_t ldb, int32_t* sums,
                                hipStream_t stream);

// One-time reorder of B (K x N, elements of elem_bytes) into K-major rows of
// ldbp elements (pack.hip). b_rowmajor: B is N-contiguous (b(k,n) = B[k*ldb+n]).
hipError_t launch_pack_b(int64_t K, int64_t N, const void* B, int64_t ldb, bool b_rowmajor,
                         int elem_bytes, void* Bp, int64_t ldbp, hipStream_t stream);

}  // namespace g355
