// C ABI of the routing of tokens to experts and of their rows' way there and
// back: argument validation and dispatch.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gemm355.h"
#include "routing.hpp"

using namespace g355;

namespace {

constexpr int64_t kMaxDim = int64_t{1} << 30;

bool valid_type(int d) { return d == GEMM_OUT_F32 || d == GEMM_OUT_BF16; }
bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
uintptr_t size_of(int d) { return d == GEMM_OUT_F32 ? 4 : 2; }

gemm_status launched(hipError_t err) { return err == hipSuccess ? GEMM_OK : GEMM_ERR_HIP; }

// Checks that gemm_route and its gradient share.
gemm_status check_route(int64_t T, int64_t E, int64_t top_k, int l_dtype, int score) {
  if (!valid_type(l_dtype) || (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID))
    return GEMM_ERR_BAD_ENUM;
  if (bad_dim(T) || E < 1 || E > kMaxDim || top_k < 1 || top_k > E) return GEMM_ERR_BAD_DIM;
  if (E > kMaxExperts || top_k > kMaxTopK) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Checks that the row movements share.
gemm_status check_rows(int64_t T, int64_t top_k, int64_t R, int64_t N) {
  if (bad_dim(T) || bad_dim(R) || bad_dim(N) || top_k < 1 || top_k > kMaxDim) return GEMM_ERR_BAD_DIM;
  if (top_k > kMaxSlots) return GEMM_ERR_UNSUPPORTED;
  if (T * top_k > kMaxDim) return GEMM_ERR_BAD_DIM;
  return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status gemm_route(int64_t T, int64_t E, int64_t top_k, const void* logits, int64_t ldl,
                       gemm_out_dtype l_dtype, gemm_score score, const float* bias,
                       int64_t groups, int64_t top_groups, int group_best, int renormalise,
                       float scale, int32_t* expert, float* weight, void* stream) {
  const gemm_status st = check_route(T, E, top_k, l_dtype, score);
  if (st != GEMM_OK) return st;
  if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      (group_best != 1 && group_best != 2) || top_k > E / groups * top_groups)
    return GEMM_ERR_BAD_DIM;
  if (groups > kMaxRouteGroups) return GEMM_ERR_UNSUPPORTED;
  if (ldl < E) return GEMM_ERR_BAD_LD;
  if (T == 0) return GEMM_OK;
  if (logits == nullptr || expert == nullptr || weight == nullptr) return GEMM_ERR_NULL_POINTER;
  if (!aligned(logits, size_of(l_dtype)) || !aligned(bias, 4) || !aligned(expert, 4) || !aligned(weight, 4))
    return GEMM_ERR_UNSUPPORTED;
  RouteArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.bias = bias;
  a.expert = expert;
  a.weight = weight;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.top_k = static_cast<int>(top_k);
  a.sigmoid = score == GEMM_SCORE_SIGMOID;
  a.renormalise = renormalise != 0;
  a.groups = static_cast<int>(groups);
  a.top_groups = static_cast<int>(top_groups);
  a.group_best = group_best;
  a.scale = scale;
  (void)hipGetLastError();  // an earlier call's pending error is not this call's
  return launched(launch_route(a, l_dtype == GEMM_OUT_BF16, static_cast<hipStream_t>(stream)));
}

gemm_status gemm_route_grad(int64_t T, int64_t E, int64_t top_k, const void* logits, int64_t ldl,
                            gemm_out_dtype l_dtype, gemm_score score, int renormalise, float scale,
                            const int32_t* expert, const float* dweight, void* dlogits,
                            int64_t ldd, void* stream) {
  const gemm_status st = check_route(T, E, top_k, l_dtype, score);
  if (st != GEMM_OK) return st;
  if (ldl < E || ldd < E) return GEMM_ERR_BAD_LD;
  if (T == 0) return GEMM_OK;
  if (logits == nullptr || expert == nullptr || dweight == nullptr || dlogits == nullptr)
    return GEMM_ERR_NULL_POINTER;
  if (!aligned(logits, size_of(l_dtype)) || !aligned(dlogits, size_of(l_dtype)) || !aligned(expert, 4) ||
      !aligned(dweight, 4))
    return GEMM_ERR_UNSUPPORTED;
  RouteGradArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.expert = expert;
  a.dweight = dweight;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.top_k = static_cast<int>(top_k);
  a.sigmoid = score == GEMM_SCORE_SIGMOID;
  a.renormalise = renormalise != 0;
  a.scale = scale;
  (void)hipGetLastError();
  return launched(launch_route_grad(a, l_dtype == GEMM_OUT_BF16, static_cast<hipStream_t>(stream)));
}

size_t gemm_route_order_workspace_size(int64_t S, int64_t G) {
  if (S <= 0 || S > kMaxDim || G < 0 || G > kMaxOrderGroups || order_small(S, G)) return 0;
  int chunk, chunks;
  order_chunks(S, G, chunk, chunks);
  return static_cast<size_t>(chunks) * (G + 1) * sizeof(int32_t);
}

gemm_status gemm_route_order(int64_t S, int64_t G, const int32_t* expert, int32_t* offsets,
                             int32_t* position, int32_t* order, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (bad_dim(S) || G < 0) return GEMM_ERR_BAD_DIM;
  if (G > kMaxOrderGroups) return GEMM_ERR_UNSUPPORTED;
  if (offsets == nullptr || (S > 0 && (expert == nullptr || position == nullptr))) return GEMM_ERR_NULL_POINTER;
  const size_t need = gemm_route_order_workspace_size(S, G);
  if (need > 0 && workspace == nullptr) return GEMM_ERR_NULL_POINTER;
  if (workspace_bytes < need) return GEMM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(expert, 4) || !aligned(offsets, 4) || !aligned(position, 4) || !aligned(order, 4) ||
      !aligned(workspace, 4))
    return GEMM_ERR_UNSUPPORTED;
  OrderArgs a{};
  a.expert = expert;
  a.offsets = offsets;
  a.position = position;
  a.order = order;
  a.counts = static_cast<int32_t*>(workspace);
  a.S = static_cast<int>(S);
  a.G = static_cast<int>(G);
  order_chunks(S, G, a.chunk, a.chunks);
  (void)hipGetLastError();
  return launched(launch_order(a, static_cast<hipStream_t>(stream)));
}

gemm_status gemm_dispatch_rows(int64_t T, int64_t top_k, int64_t R, int64_t N, const void* X,
                               int64_t ldx, int elem_bytes, const int32_t* position, void* Y,
                               int64_t ldy, void* stream) {
  if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return GEMM_ERR_BAD_ENUM;
  const gemm_status st = check_rows(T, top_k, R, N);
  if (st != GEMM_OK) return st;
  if (ldx < std::max<int64_t>(1, N) || ldy < std::max<int64_t>(1, N)) return GEMM_ERR_BAD_LD;
  if (T == 0 || R == 0 || N == 0) return GEMM_OK;
  if (X == nullptr || Y == nullptr || position == nullptr) return GEMM_ERR_NULL_POINTER;
  if (!aligned(X, elem_bytes) || !aligned(Y, elem_bytes) || !aligned(position, 4)) return GEMM_ERR_UNSUPPORTED;
  RowsArgs a{};
  a.from = X;
  a.ld_from = ldx;
  a.to = Y;
  a.ld_to = ldy;
  a.position = position;
  a.T = static_cast<int>(T);
  a.top_k = static_cast<int>(top_k);
  a.R = static_cast<int>(R);
  a.N = static_cast<int>(N);
  (void)hipGetLastError();
  return launched(launch_dispatch(a, elem_bytes, static_cast<hipStream_t>(stream)));
}

gemm_status gemm_combine_rows(int64_t T, int64_t top_k, int64_t R, int64_t N, const void* Y,
                              int64_t ldy, gemm_out_dtype y_dtype, const int32_t* position,
                              const float* weight, float beta, void* C, int64_t ldc,
                              gemm_out_dtype c_dtype, void* stream) {
  if (!valid_type(y_dtype) || !valid_type(c_dtype)) return GEMM_ERR_BAD_ENUM;
  const gemm_status st = check_rows(T, top_k, R, N);
  if (st != GEMM_OK) return st;
  if (ldy < std::max<int64_t>(1, N) || ldc < std::max<int64_t>(1, N)) return GEMM_ERR_BAD_LD;
  if (T == 0 || N == 0) return GEMM_OK;
  if (C == nullptr || position == nullptr || (R > 0 && Y == nullptr)) return GEMM_ERR_NULL_POINTER;
  if (!aligned(Y, size_of(y_dtype)) || !aligned(C, size_of(c_dtype)) || !aligned(position, 4) ||
      !aligned(weight, 4))
    return GEMM_ERR_UNSUPPORTED;
  RowsArgs a{};
  a.from = Y;
  a.ld_from = ldy;
  a.to = C;
  a.ld_to = ldc;
  a.position = position;
  a.weight = weight;
  a.T = static_cast<int>(T);
  a.top_k = static_cast<int>(top_k);
  a.R = static_cast<int>(R);
  a.N = static_cast<int>(N);
  a.beta = beta;
  (void)hipGetLastError();
  return launched(launch_combine(a, y_dtype == GEMM_OUT_BF16, c_dtype == GEMM_OUT_BF16,
                                 static_cast<hipStream_t>(stream)));
}

gemm_status gemm_combine_rows_grad(int64_t T, int64_t top_k, int64_t R, int64_t N, const void* D,
                                   int64_t ldd, gemm_out_dtype d_dtype, const void* Y, int64_t ldy,
                                   gemm_out_dtype y_dtype, const int32_t* position,
                                   const float* weight, void* dY, int64_t lddy, float* dweight,
                                   void* stream) {
  if (!valid_type(d_dtype) || !valid_type(y_dtype)) return GEMM_ERR_BAD_ENUM;
  const gemm_status st = check_rows(T, top_k, R, N);
  if (st != GEMM_OK) return st;
  const int64_t least = std::max<int64_t>(1, N);
  if (ldd < least || lddy < least || (dweight != nullptr && ldy < least)) return GEMM_ERR_BAD_LD;
  if (T == 0) return GEMM_OK;
  if (position == nullptr) return GEMM_ERR_NULL_POINTER;
  if (N > 0 && R > 0 && (D == nullptr || dY == nullptr || (dweight != nullptr && Y == nullptr)))
    return GEMM_ERR_NULL_POINTER;
  if (dweight == nullptr && (N == 0 || R == 0)) return GEMM_OK;
  if (!aligned(D, size_of(d_dtype)) || !aligned(Y, size_of(y_dtype)) || !aligned(dY, size_of(y_dtype)) ||
      !aligned(position, 4) || !aligned(weight, 4) || !aligned(dweight, 4))
    return GEMM_ERR_UNSUPPORTED;
  RowsArgs a{};
  a.from = D;
  a.ld_from = ldd;
  a.y = Y;
  a.ldy = ldy;
  a.to = dY;
  a.ld_to = lddy;
  a.position = position;
  a.weight = weight;
  a.dweight = dweight;
  a.T = static_cast<int>(T);
  a.top_k = static_cast<int>(top_k);
  a.R = static_cast<int>(R);
  a.N = static_cast<int>(N);
  (void)hipGetLastError();
  return launched(launch_combine_grad(a, d_dtype == GEMM_OUT_BF16, y_dtype == GEMM_OUT_BF16,
                                      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
