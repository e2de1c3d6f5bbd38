// Rows of tokens to their experts and back. The formulas are in gemm355.h.
//
// Everything here is bound by memory. Work is laid out by token, so that a
// token's own row (X, C or D) passes through HBM once, whatever top_k is.

#include "common.hpp"
#include "routing.hpp"

namespace g355 {

namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16_bits(v);
  else static_cast<float*>(p)[i] = v;
}

}  // namespace

template <class E>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(RowsArgs p) {
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
  const E* from = static_cast<const E*>(p.from) + t * p.ld_from;
  E* to = static_cast<E*>(p.to);
  const int32_t* position = p.position + t * p.top_k;
  for (int n = blockIdx.y * kThreads + threadIdx.x; n < p.N; n += gridDim.y * kThreads) {
    const E v = from[n];
    for (int j = 0; j < p.top_k; ++j) {
      const int r = position[j];
      if (r >= 0 && r < p.R) to[r * p.ld_to + n] = v;
    }
  }
  }
}

template <bool YB, bool CB>
__global__ void __launch_bounds__(kThreads) combine_kernel(RowsArgs p) {
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
  const int32_t* position = p.position + t * p.top_k;
  const float* weight = p.weight ? p.weight + t * p.top_k : nullptr;
  for (int n = blockIdx.y * kThreads + threadIdx.x; n < p.N; n += gridDim.y * kThreads) {
    float v = p.beta != 0.f ? p.beta * load1<CB>(p.to, t * p.ld_to + n) : 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      const int r = position[j];
      if (r >= 0 && r < p.R) v = fmaf(weight ? weight[j] : 1.f, load1<YB>(p.from, r * p.ld_from + n), v);
    }
    store1<CB>(p.to, t * p.ld_to + n, v);
  }
  }
}

template <bool DB, bool YB>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(RowsArgs p) {
  __shared__ float part[kThreads / 64];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
  const int32_t* position = p.position + t * p.top_k;
  for (int j = 0; j < p.top_k; ++j) {
    const int r = position[j];
    const bool live = r >= 0 && r < p.R;
    const float w = p.weight ? p.weight[t * p.top_k + j] : 1.f;
    float dot = 0.f;
    if (live) {
      for (int n = threadIdx.x; n < p.N; n += kThreads) {
        const float d = load1<DB>(p.from, t * p.ld_from + n);
        store1<YB>(p.to, r * p.ld_to + n, w * d);
        if (p.dweight) dot = fmaf(d, load1<YB>(p.y, r * p.ldy + n), dot);
      }
    }
    if (p.dweight) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
      __syncthreads();
      if (threadIdx.x == 0) p.dweight[t * p.top_k + j] = (part[0] + part[1]) + (part[2] + part[3]);
      __syncthreads();
    }
  }
  }
}

hipError_t launch_dispatch(const RowsArgs& a, int elem_bytes, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.T < kMaxGrid ? a.T : kMaxGrid), 1), block(kThreads);
  if (elem_bytes == 1) hipLaunchKernelGGL(dispatch_kernel<uint8_t>, grid, block, 0, stream, a);
  else if (elem_bytes == 2) hipLaunchKernelGGL(dispatch_kernel<uint16_t>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(dispatch_kernel<uint32_t>, grid, block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_combine(const RowsArgs& a, bool y_bf16, bool c_bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.T < kMaxGrid ? a.T : kMaxGrid), 1), block(kThreads);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  if (y_bf16) c_bf16 ? go(combine_kernel<true, true>) : go(combine_kernel<true, false>);
  else c_bf16 ? go(combine_kernel<false, true>) : go(combine_kernel<false, false>);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const RowsArgs& a, bool d_bf16, bool y_bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.T < kMaxGrid ? a.T : kMaxGrid)), block(kThreads);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  if (d_bf16) y_bf16 ? go(combine_grad_kernel<true, true>) : go(combine_grad_kernel<true, false>);
  else y_bf16 ? go(combine_grad_kernel<false, true>) : go(combine_grad_kernel<false, false>);
  return hipGetLastError();
}

}  // namespace g355
