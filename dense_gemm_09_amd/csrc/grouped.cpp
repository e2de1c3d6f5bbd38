// C ABI of the products grouped by rows (one weight per group of tokens) and
// of their weight gradient: argument validation, plan and dispatch.
//
// The groups' row ranges are device data (they come out of a router on the
// GPU), so everything here is decided from what the host knows: the number of
// groups, the rows in all, and the sizes of a weight. The kernels find each
// workgroup's group themselves (grouping.hpp).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gemm355.h"
#include "grouped_plan.hpp"
#include "internal.hpp"
#include "row_copies.hpp"

using namespace g355;

namespace {

constexpr int64_t kMaxDim = int64_t{1} << 30;
constexpr int64_t kMaxGroups = int64_t{1} << 16;
constexpr int64_t k2G = int64_t{1} << 31;

bool valid_layout(int l) { return l == GEMM_ROW_MAJOR || l == GEMM_COL_MAJOR; }
bool valid_out(int d) { return d == GEMM_OUT_F32 || d == GEMM_OUT_BF16; }
bool valid_act(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_GELU_TANH; }
bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int c_vector(const void* C, int64_t ldc, int64_t stride, int c_dtype) {
  return aligned(C, c_dtype == GEMM_OUT_F32 ? 16 : 8) && ldc % 4 == 0 && stride % 4 == 0 ? 1 : 0;
}

struct Scales {
  const float* a;
  const int32_t* zero_a;
  const float* b;
  const int32_t* sum_b;
};

gemm_status run_grouped(ElemType type, int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                        const void* A, int64_t lda, const int32_t* offsets, const void* B,
                        int64_t ldb, int layout_b, int64_t stride_b, const Scales& sc, float beta,
                        void* C, int64_t ldc, int c_dtype, const void* bias, int act,
                        void* stream) {
  const bool bytes1 = type != TY_BF16;
  if (!valid_layout(layout_b) || !valid_out(c_dtype) || !valid_act(act)) return GEMM_ERR_BAD_ENUM;
  if (bad_dim(T) || bad_dim(N) || bad_dim(K) || G < 0 || G > kMaxGroups) return GEMM_ERR_BAD_DIM;
  const bool b_kmajor = layout_b == GEMM_COL_MAJOR;
  if (bytes1 && !b_kmajor) return GEMM_ERR_UNSUPPORTED;
  if (type == TY_I8 && K > kMaxInt8K) return GEMM_ERR_UNSUPPORTED;
  if (lda < std::max<int64_t>(1, K) || ldb < std::max<int64_t>(1, b_kmajor ? K : N) ||
      ldc < std::max<int64_t>(1, N) || stride_b < 0)
    return GEMM_ERR_BAD_LD;
  if (G == 0 || T == 0 || N == 0) return GEMM_OK;
  if (C == nullptr || offsets == nullptr) return GEMM_ERR_NULL_POINTER;
  if (K > 0 && (A == nullptr || B == nullptr)) return GEMM_ERR_NULL_POINTER;
  if (bytes1 && (sc.a == nullptr || sc.b == nullptr)) return GEMM_ERR_NULL_POINTER;
  if ((sc.zero_a == nullptr) != (sc.sum_b == nullptr)) return GEMM_ERR_NULL_POINTER;
  if (!aligned(offsets, 4)) return GEMM_ERR_UNSUPPORTED;

  const int64_t es = bytes1 ? 1 : 2, ce = 16 / es;
  GroupedPlan plan = plan_grouped(G, T, N, !b_kmajor);
  LaunchSpec spec{};
  spec.fp8 = type == TY_FP8;
  spec.i8 = type == TY_I8;
  spec.out = c_dtype == GEMM_OUT_F32 ? OUT_F32 : OUT_BF16;
  spec.a_kmajor = true;
  spec.b_kmajor = b_kmajor;
  // DMA: 32-bit offsets into a tile's rows of A and into one group's weight, and
  // 32-bit row distances where the copies follow the rows.
  const int64_t b_last = b_kmajor ? (N - 1) * ldb + K - 1 : (K - 1) * ldb + N - 1;
  const bool a_ok = (256 * lda + K) * es < k2G && (bytes1 || aligned(A, 2));
  const bool b_ok = (b_last + 1) * es + 2 < k2G &&
                    (b_kmajor ? bytes1 || aligned(B, 2)
                              : ldb < k2G && rows_dma_ok(reinterpret_cast<uintptr_t>(B), ldb, stride_b,
                                                         (G - 1) * stride_b + b_last));
  spec.loader_a = spec.loader_b = LOAD_GENERIC;
  if (K == 0 || (a_ok && b_ok)) {
    spec.loader_a = LOAD_DIRECT;
    spec.loader_b = b_kmajor || K == 0 ? LOAD_DIRECT : LOAD_DIRECT_N;
    spec.ragged = K % ce != 0;
  } else {
    plan = {128, 128, most_row_tiles(G, T, 128) * ceil_div(N, 128)};
  }
  if (plan.grid > INT32_MAX) return GEMM_ERR_BAD_DIM;

  GemmArgs a{};
  a.A = A;
  a.B = B;
  a.C = C;
  a.bias = static_cast<const uint16_t*>(bias);
  a.scale_a = sc.a;
  a.scale_b = sc.b;
  a.zero_a = sc.zero_a;
  a.sum_b = sc.sum_b;
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldc;
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.alpha = alpha;
  a.beta = beta;
  a.act = act;
  a.b_mn_major = b_kmajor ? 0 : 1;
  a.c_vec = c_vector(C, ldc, 0, c_dtype);
  a.split_k = 1;
  a.k_split_len = static_cast<int>(std::max<int64_t>(1, K));
  a.tiles_n = static_cast<int>(ceil_div(N, plan.bn));
  a.offsets = offsets;
  a.groups = static_cast<int>(G);
  a.rows_total = static_cast<int>(T);
  a.stride_b = stride_b;
  (void)hipGetLastError();  // an earlier call's pending error is not this call's
  const auto s = static_cast<hipStream_t>(stream);
  hipError_t err;
  if (plan.bm == 256)
    err = spec.i8    ? launch_turn_i8(spec, plan.grid, a, s)
          : spec.fp8 ? launch_turn_fp8(spec, plan.grid, a, s)
                     : launch_turn_bf16(spec, plan.grid, a, s);
  else if (c_dtype == GEMM_OUT_F32)
    err = spec.ragged ? launch_grouped_r1_p1(plan, spec, a, s) : launch_grouped_r0_p1(plan, spec, a, s);
  else
    err = spec.ragged ? launch_grouped_r1_p2(plan, spec, a, s) : launch_grouped_r0_p2(plan, spec, a, s);
  return err == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // namespace

extern "C" {

gemm_status gemm_grouped_bf16(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                              const void* A, int64_t lda, const int32_t* offsets, const void* B,
                              int64_t ldb, gemm_layout layout_b, int64_t stride_b, float beta,
                              void* C, int64_t ldc, gemm_out_dtype c_dtype, const void* bias,
                              gemm_act act, void* stream) {
  return run_grouped(TY_BF16, G, T, N, K, alpha, A, lda, offsets, B, ldb, layout_b, stride_b,
                     Scales{}, beta, C, ldc, c_dtype, bias, act, stream);
}

gemm_status gemm_grouped_fp8_scaled(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                                    const void* A, int64_t lda, const int32_t* offsets,
                                    const void* B, int64_t ldb, gemm_layout layout_b,
                                    int64_t stride_b, const float* scale_a, const float* scale_b,
                                    float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                                    const void* bias, gemm_act act, void* stream) {
  return run_grouped(TY_FP8, G, T, N, K, alpha, A, lda, offsets, B, ldb, layout_b, stride_b,
                     Scales{scale_a, nullptr, scale_b, nullptr}, beta, C, ldc, c_dtype, bias, act,
                     stream);
}

gemm_status gemm_grouped_int8_scaled(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                                     const void* A, int64_t lda, const int32_t* offsets,
                                     const void* B, int64_t ldb, gemm_layout layout_b,
                                     int64_t stride_b, const float* scale_a,
                                     const int32_t* zero_a, const float* scale_b,
                                     const int32_t* sum_b, float beta, void* C, int64_t ldc,
                                     gemm_out_dtype c_dtype, const void* bias, gemm_act act,
                                     void* stream) {
  return run_grouped(TY_I8, G, T, N, K, alpha, A, lda, offsets, B, ldb, layout_b, stride_b,
                     Scales{scale_a, zero_a, scale_b, sum_b}, beta, C, ldc, c_dtype, bias, act,
                     stream);
}

gemm_status gemm_grouped_bf16_wgrad(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                                    const void* D, int64_t ldd, const void* X, int64_t ldx,
                                    const int32_t* offsets, float beta, void* C, int64_t ldc,
                                    int64_t stride_c, gemm_out_dtype c_dtype, void* stream) {
  if (!valid_out(c_dtype)) return GEMM_ERR_BAD_ENUM;
  if (bad_dim(T) || bad_dim(N) || bad_dim(K) || G < 0 || G > kMaxGroups) return GEMM_ERR_BAD_DIM;
  if (ldd < std::max<int64_t>(1, N) || ldx < std::max<int64_t>(1, K) ||
      ldc < std::max<int64_t>(1, K))
    return GEMM_ERR_BAD_LD;
  if (G == 0 || N == 0 || K == 0) return GEMM_OK;
  // Every group's gradient is written: they may not overlap.
  if (stride_c < 0 || (G > 1 && stride_c < (N - 1) * ldc + K)) return GEMM_ERR_BAD_LD;
  if (C == nullptr || offsets == nullptr) return GEMM_ERR_NULL_POINTER;
  if (T > 0 && (D == nullptr || X == nullptr)) return GEMM_ERR_NULL_POINTER;
  if (!aligned(offsets, 4)) return GEMM_ERR_UNSUPPORTED;

  GroupedPlan plan = plan_wgrad(G, N, K);
  LaunchSpec spec{};
  spec.out = c_dtype == GEMM_OUT_F32 ? OUT_F32 : OUT_BF16;
  // DMA: 32-bit offsets into the 64 rows of a slice.
  const bool dma = T == 0 || (128 * std::max(ldd, ldx) < k2G &&
                              rows_dma_ok(reinterpret_cast<uintptr_t>(D), ldd, 0, (T - 1) * ldd + N - 1) &&
                              rows_dma_ok(reinterpret_cast<uintptr_t>(X), ldx, 0, (T - 1) * ldx + K - 1));
  spec.loader_a = spec.loader_b = dma ? LOAD_ROWS : LOAD_GENERIC;
  if (!dma) {
    const int64_t tiles = ceil_div(N, 128) * ceil_div(K, 128);
    plan = {128, 128, G * (tiles >= kWgradXcdTiles ? 8 * ceil_div(tiles, 8) : tiles)};
  }
  if (plan.grid > INT32_MAX) return GEMM_ERR_BAD_DIM;

  GemmArgs a{};
  a.A = D;
  a.B = X;
  a.C = C;
  a.lda = ldd;
  a.ldb = ldx;
  a.ldc = ldc;
  a.M = static_cast<int>(N);
  a.N = static_cast<int>(K);
  a.alpha = alpha;
  a.beta = beta;
  a.a_mn_major = a.b_mn_major = 1;
  a.c_vec = c_vector(C, ldc, G > 1 ? stride_c : 0, c_dtype);
  a.split_k = 1;
  a.tiles_m = static_cast<int>(ceil_div(N, plan.bm));
  a.tiles_n = static_cast<int>(ceil_div(K, plan.bn));
  a.offsets = offsets;
  a.groups = static_cast<int>(G);
  a.rows_total = static_cast<int>(T);
  a.stride_b = stride_c;
  (void)hipGetLastError();
  const auto s = static_cast<hipStream_t>(stream);
  const hipError_t err = plan.bm == 256             ? launch_turn_wgrad(spec, plan.grid, a, s)
                         : c_dtype == GEMM_OUT_F32 ? launch_wgrad_p1(plan, spec, a, s)
                                                   : launch_wgrad_p2(plan, spec, a, s);
  return err == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
