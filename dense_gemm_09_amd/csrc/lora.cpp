// C ABI of the projection with low-rank adapters: argument validation, plan and dispatch.
//
// Two to four launches: the first factors' product h (with the sum of its shares of K
// where it has several and the tiles run), and the projection's own kernel, which adds
// h times the second factors to its accumulators before its epilogue (with the
// reduction of a split K).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gemm355.h"
#include "internal.hpp"
#include "lora.hpp"

using namespace g355;

namespace {

constexpr int64_t kMaxDim = int64_t{1} << 30;
constexpr int64_t k2G = int64_t{1} << 31;

bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }
// Whether rows of K BF16 elements, ld apart, span less than 2 GiB. (A product of a
// leading dimension that nothing bounds is not formed: it may exceed 64 bits.)
bool under_2g(int64_t rows, int64_t K, int64_t ld) {
  if (rows > 1 && ld >= k2G / 2 / (rows - 1) + 1) return false;
  return ((rows - 1) * ld + K) * 2 < k2G;
}
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows up to which the kernels for few rows (gemm_skinny.hip) are used; what they and
// the tiles measure is there.
constexpr int64_t kFewRows = 16;

// The workspace: h, its partial sums, the product's partial sums of a split K.
size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t h_bytes(int64_t M, int64_t R) { return rounded(static_cast<size_t>(M) * 2 * kMostParts * padded_rank(R)); }
size_t partial_bytes(int64_t M, int64_t K, int64_t R) {
  const int shares = lora_shares(M, K, R).shares;
  return shares == 1 && M > kFewRows ? 0 : rounded(static_cast<size_t>(shares) * M * padded_rank(R) * sizeof(float));
}

}  // namespace

hipError_t g355::launch_lora(const Plan& plan, const LaunchSpec& spec, const LoraArgs& args, hipStream_t stream) {
  using Fn = hipError_t (*)(const Plan&, const LoraArgs&, hipStream_t);
  static constexpr Fn kParts[2][3] = {{launch_lora_r0_p0, launch_lora_r0_p1, launch_lora_r0_p2},
                                      {launch_lora_r1_p0, launch_lora_r1_p1, launch_lora_r1_p2}};
  const int part = plan.split > 1 ? PART_SPLIT : spec.out == OUT_F32 ? PART_F32 : PART_BF16;
  return kParts[spec.ragged ? 1 : 0][part](plan, args, stream);
}

extern "C" {

size_t gemm_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R) {
  if (M <= 0 || N <= 0 || bad_dim(M) || bad_dim(N) || bad_dim(K) || R < 0 || R > kMaxRank) return 0;
  return h_bytes(M, R) + partial_bytes(M, K, R) + make_tile_plan(M, N, K, false).workspace;
}

gemm_status gemm_lora_bf16(int64_t M, int64_t N, int64_t K, int64_t G, int64_t R, float alpha,
                           const void* A, int64_t lda, const void* B, int64_t ldb,
                           const int32_t* adapter, const void* down, int64_t ld_down,
                           int64_t stride_down, const void* up, int64_t ld_up, int64_t stride_up,
                           const float* scale, float beta, void* C, int64_t ldc,
                           gemm_out_dtype c_dtype, const void* bias, gemm_act act,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if ((c_dtype != GEMM_OUT_F32 && c_dtype != GEMM_OUT_BF16) || act < GEMM_ACT_NONE ||
      act > GEMM_ACT_GELU_TANH)
    return GEMM_ERR_BAD_ENUM;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K) || G < 0 || R < 0) return GEMM_ERR_BAD_DIM;
  if (R > kMaxRank || G > kMaxAdapters) return GEMM_ERR_UNSUPPORTED;
  const bool adapters = G > 0 && R > 0;
  if (lda < std::max<int64_t>(1, K) || ldb < std::max<int64_t>(1, K) || ldc < std::max<int64_t>(1, N))
    return GEMM_ERR_BAD_LD;
  if (adapters && (ld_down < std::max<int64_t>(1, K) || ld_up < R || stride_down < 0 || stride_up < 0))
    return GEMM_ERR_BAD_LD;
  if (M == 0 || N == 0) return GEMM_OK;
  if (C == nullptr || (K > 0 && (A == nullptr || B == nullptr))) return GEMM_ERR_NULL_POINTER;
  if (adapters && (adapter == nullptr || up == nullptr || (K > 0 && down == nullptr)))
    return GEMM_ERR_NULL_POINTER;
  const size_t need = gemm_lora_workspace_size(M, N, K, R);
  if (need > 0 && workspace == nullptr) return GEMM_ERR_NULL_POINTER;
  if (workspace_bytes < need) return GEMM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16) || !aligned(adapter, 4) || !aligned(scale, 4) || !aligned(down, 2) ||
      !aligned(up, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(bias, 2) ||
      !aligned(C, c_dtype == GEMM_OUT_F32 ? 4 : 2))
    return GEMM_ERR_UNSUPPORTED;
  // The kernels for few rows read rows of 16 bytes at a time. The one that does not
  // stream has a workgroup of 1024 threads for every 16 columns, and HIP counts a launch's
  // threads in 32 bits: more columns run on tiles. They address the weight in 64 bits,
  // the tiles' copies both operands in 32.
  const bool few = M <= kFewRows && K % 8 == 0 && lda % 8 == 0 && ldb % 8 == 0 && ldb < k2G && aligned(A, 16) &&
                   aligned(B, 16) && (skinny_streams_lora(K, padded_rank(R)) || (N + 15) / 16 < int64_t{1} << 22);
  if (!under_2g(M, K, lda) || (!few && !under_2g(N, K, ldb))) return GEMM_ERR_UNSUPPORTED;

  Plan plan = make_tile_plan(M, N, K, false);
  // Tiles of 128x128 that the dense product splits in two and that the CUs hold at
  // once take two groups of waves along K in one workgroup instead: no partial sums.
  // BF16 output, split in two -> two groups: 777 x 4093 x 4099 90 -> 79 us, 1024 x 4096 x
  // 4096 61 -> 56, 512 x 8192 x 4096 60 -> 53, 777 x 4096 x 4096 55 -> 54; the other way
  // for 1500 x 2048 x 4096 (192 tiles) 55 -> 56 and 1100 x 3584 x 7168 86 -> 88.
  const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128);
  if (plan.bm == 128 && plan.split == 2 && tiles <= 256) {
    plan.split = 1;
    plan.k_split_len = static_cast<int>((K + plan.bk - 1) / plan.bk * plan.bk);
    plan.grid = tiles;
  }
  if (plan.grid > INT32_MAX) return GEMM_ERR_BAD_DIM;
  const auto s = static_cast<hipStream_t>(stream);
  LoraArgs a{};
  a.A = A;
  a.B = B;
  a.C = C;
  a.bias = static_cast<const uint16_t*>(bias);
  a.workspace = reinterpret_cast<float*>(static_cast<char*>(workspace) + h_bytes(M, R) + partial_bytes(M, K, R));
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldc;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.alpha = alpha;
  a.beta = beta;
  a.act = act;
  a.c_vec = aligned(C, c_dtype == GEMM_OUT_F32 ? 16 : 8) && ldc % 4 == 0 ? 1 : 0;
  a.ws_vec = 1;
  a.split_k = plan.split;
  a.k_split_len = plan.k_split_len;
  a.tiles_m = static_cast<int>((M + plan.bm - 1) / plan.bm);
  a.tiles_n = static_cast<int>((N + plan.bn - 1) / plan.bn);
  a.adapter = adapter;
  a.h = static_cast<const uint16_t*>(workspace);
  a.partial = reinterpret_cast<const float*>(static_cast<char*>(workspace) + h_bytes(M, R));
  const LoraShares shares = lora_shares(M, K, R);
  a.shares = shares.shares;
  a.up = static_cast<const uint16_t*>(up);
  a.ld_up = ld_up;
  a.stride_up = stride_up;
  a.adapters = adapters ? static_cast<int>(G) : 0;
  a.rank = static_cast<int>(R);
  a.pad = static_cast<int>(padded_rank(R));
  a.parts = parts_of_h(c_dtype == GEMM_OUT_F32);
  (void)hipGetLastError();  // an earlier call's pending error is not this call's
  if (adapters) {
    LoraDownArgs d{};
    d.A = static_cast<const uint16_t*>(A);
    d.lda = lda;
    d.adapter = adapter;
    d.down = static_cast<const uint16_t*>(down);
    d.ld_down = ld_down;
    d.stride_down = stride_down;
    d.scale = scale;
    d.h = few ? nullptr : static_cast<uint16_t*>(workspace);
    d.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + h_bytes(M, R));
    d.shares = shares.shares;
    d.share_len = shares.len;
    d.M = a.M;
    d.K = a.K;
    d.adapters = a.adapters;
    d.rank = a.rank;
    d.pad = a.pad;
    d.parts = a.parts;
    if (launch_lora_down(d, s) != hipSuccess) return GEMM_ERR_HIP;
  }
  LaunchSpec spec{};
  spec.a_kmajor = spec.b_kmajor = true;
  spec.loader_a = spec.loader_b = LOAD_DIRECT;
  spec.out = c_dtype == GEMM_OUT_F32 ? OUT_F32 : OUT_BF16;
  spec.ragged = K % 8 != 0;
  if (few)
    return launch_skinny_lora(spec, a, s) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
  if (launch_lora(plan, spec, a, s) != hipSuccess) return GEMM_ERR_HIP;
  if (plan.split > 1 && launch_splitk_reduce(plan, spec, a, s) != hipSuccess) return GEMM_ERR_HIP;
  return GEMM_OK;
}

}  // extern "C"
