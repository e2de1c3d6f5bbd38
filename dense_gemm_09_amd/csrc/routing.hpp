// Host-side interface between the routing entry points and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "order_plan.hpp"

namespace g355 {

constexpr int kMaxExperts = 1024;      // logits of a row that the routing kernels hold
constexpr int kMaxTopK = 32;
constexpr int kMaxRouteGroups = 64;    // one lane each
constexpr int kMaxSlots = 64;          // top_k of the row movements (a slot per lane)

// Workgroups of a launch at most (HIP counts a launch's threads in 32 bits);
// past them, workgroups take several tokens.
constexpr int kMaxGrid = 1 << 20;

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  const float* bias;  // or nullptr
  int32_t* expert;
  float* weight;
  int T, E, top_k;
  int sigmoid, renormalise;
  int groups, top_groups, group_best;
  float scale;
};

struct RouteGradArgs {
  const void* logits;
  int64_t ldl;
  const int32_t* expert;
  const float* dweight;
  void* dlogits;
  int64_t ldd;
  int T, E, top_k;
  int sigmoid, renormalise;
  float scale;
};

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_route_grad(const RouteGradArgs& a, bool bf16, hipStream_t stream);

struct OrderArgs {
  const int32_t* expert;
  int32_t* offsets;
  int32_t* position;
  int32_t* order;  // or nullptr
  int32_t* counts; // workspace: [chunks][G + 1]
  int S, G;
  int chunk, chunks;  // slots per chunk (a multiple of 64 per wave)
};

hipError_t launch_order(const OrderArgs& a, hipStream_t stream);

struct RowsArgs {
  const void* from;   // dispatch: X; combine: Y; combine's gradient: D
  int64_t ld_from;
  const void* y;      // combine's gradient: Y
  int64_t ldy;
  void* to;           // dispatch: Y; combine: C; combine's gradient: dY
  int64_t ld_to;
  const int32_t* position;
  const float* weight;  // or nullptr: ones
  float* dweight;       // or nullptr
  int T, top_k, R, N;
  float beta;
};

hipError_t launch_dispatch(const RowsArgs& a, int elem_bytes, hipStream_t stream);
hipError_t launch_combine(const RowsArgs& a, bool y_bf16, bool c_bf16, hipStream_t stream);
hipError_t launch_combine_grad(const RowsArgs& a, bool d_bf16, bool y_bf16, hipStream_t stream);

}  // namespace g355
