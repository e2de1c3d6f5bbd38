// The first factor of low-rank adapters: h[m] = scale[a] * (A[m] down_a), a = adapter[m].

#include "lora.hpp"

namespace g355 {

namespace {

constexpr int kThreads = 256;

// h as two BF16 values (LoraArgs). Beyond BF16's range the second is left out:
// the difference would be NaN.
__device__ __forceinline__ void store_h(const LoraDownArgs& p, int m, int r, float h) {
  uint16_t* row = p.h + static_cast<int64_t>(m) * 2 * p.pad;
  const uint16_t high = f32_to_bf16_bits(h);
  const float rest = h - bf16_bits_to_f32(high);
  row[r] = high;
  row[p.pad + r] = (high & 0x7f80u) == 0x7f80u ? 0 : f32_to_bf16_bits(rest);
}

}  // namespace

// One wave per element of h.
__global__ void __launch_bounds__(kThreads) lora_down_kernel(LoraDownArgs p) {
  const int lane = threadIdx.x & 63;
  for (int m = blockIdx.x; m < p.M; m += gridDim.x) {
  const int r = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6);
  const int a = p.adapter[m];
  float h = 0.f;
  if (a >= 0 && a < p.adapters && r < p.rank) {
    const uint16_t* x = p.A + m * p.lda;
    const uint16_t* w = p.down + a * p.stride_down + r * p.ld_down;
    for (int k = lane; k < p.K; k += 64) h = fmaf(bf16_bits_to_f32(x[k]), bf16_bits_to_f32(w[k]), h);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) h += __shfl_xor(h, o);
    if (p.scale) h *= p.scale[a];
  }
  if (lane == 0) store_h(p, m, r, h);
  }
}

hipError_t launch_lora_down(const LoraDownArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.M < (1 << 20) ? a.M : 1 << 20), static_cast<unsigned>(a.pad / (kThreads / 64)));
  hipLaunchKernelGGL(lora_down_kernel, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace g355
