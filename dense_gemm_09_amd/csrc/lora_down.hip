// The first factor of low-rank adapters: h[m] = scale[a] * (A[m] down_a), a = adapter[m].
//
// A workgroup has 16 rows and RT times 16 ranks; its 16 waves take K in turns of 64
// elements (a whole 128-byte line of every row), with all of a wave's loads of several
// turns in flight: with K = 4096 that is one trip to memory. Rows and ranks are
// one v_mfma_f32_16x16x32_bf16's, read straight into its operands; every row is
// multiplied with every adapter that the 16 rows have, and keeps its own. (A
// product's row depends on that row of A alone, so nothing passes between requests.)
// The waves' sums are added in LDS in the order of the waves.
//
// Bound by its reads: A once for every 32 ranks, and each tile's adapters. Where
// there are few rows, ranks (RT = 1) and adapters (blockIdx.z) go to workgroups of their
// own: 64 rows of 24 adapters, K = 14336, R = 64: 72 us by a wave per element, @@ so.

#include "lora.hpp"

namespace g355 {

namespace {

constexpr int kWaves = 16;
constexpr int kTurn = 64;  // K elements of a wave's turn
constexpr int kMaxTiles = 1 << 20;

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

template <int RT>
__global__ void __launch_bounds__(64 * kWaves) lora_down_kernel(LoraDownArgs p) {
  constexpr int AHEAD = 4 / RT;  // turns whose loads are in flight
  __shared__ __attribute__((aligned(16))) float part[kWaves][RT][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane & 15, quarter = lane >> 4;
  const int r0 = blockIdx.y * 16 * RT;
  const int tiles = (p.M + 15) / 16;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int m = tile * 16 + l;
    int id = m < p.M ? p.adapter[m] : -1;
    id = id < p.adapters ? id : -1;
    const uint16_t* x = p.A + min(m, p.M - 1) * p.lda;
    unsigned left = static_cast<unsigned>(__ballot(id >= 0)) & 0xffffu;
    for (int turn = 0; left != 0; ++turn) {
      const int g = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
      const unsigned rows = static_cast<unsigned>(__ballot(id == g)) & 0xffffu;
      left &= ~rows;
      if (turn % static_cast<int>(gridDim.z) != static_cast<int>(blockIdx.z)) continue;

      const uint16_t* w[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t)
        w[t] = p.down + g * p.stride_down + min(r0 + 16 * t + l, p.rank - 1) * p.ld_down;
      f32x4 acc[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int k0 = wave * kTurn; k0 < p.K; k0 += kWaves * kTurn * AHEAD) {
        i32x4 xv[AHEAD][2], wv[AHEAD][2][RT];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int k = k0 + u * kWaves * kTurn + 32 * s + 8 * quarter;
            xv[u][s] = load8(x, k, p.K);
#pragma unroll
            for (int t = 0; t < RT; ++t) wv[u][s][t] = load8(w[t], k, p.K);
          }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < RT; ++t)
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[u][s]),
                                                               __builtin_bit_cast(bf16x8, wv[u][s][t]), acc[t], 0, 0, 0);
      }
      // Element e of lane l: row 4 (l / 16) + e, rank l % 16.
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][t][(4 * quarter + e) * 16 + l] = acc[t][e];
      __syncthreads();
      if (tid < 256 * RT) {
        const int t = tid >> 8, i = tid & 255, row = i >> 4, r = r0 + 16 * t + (i & 15);
        if (((rows >> row) & 1) && r < p.pad) {
          float h = part[0][t][i];
#pragma unroll
          for (int v = 1; v < kWaves; ++v) h += part[v][t][i];
          // Ranks past the last repeat it above, and are zeros in h.
          store_h(p, tile * 16 + row, r, r < p.rank ? (p.scale ? h * p.scale[g] : h) : 0.f);
        }
      }
      __syncthreads();
    }
  }
}

hipError_t launch_lora_down(const LoraDownArgs& a, hipStream_t stream) {
  const int tiles = (a.M + 15) / 16;
  // 32 ranks to a workgroup where the row tiles alone fill the card.
  const int rt = a.pad > 16 && tiles >= 256 ? 2 : 1;
  const int ranks = (a.pad + 16 * rt - 1) / (16 * rt);
  const int wgs = (tiles < kMaxTiles ? tiles : kMaxTiles) * ranks;
  const int shares = wgs >= 512 ? 1 : 512 / wgs < 16 ? 512 / wgs : 16;
  const dim3 grid(static_cast<unsigned>(tiles < kMaxTiles ? tiles : kMaxTiles), static_cast<unsigned>(ranks),
                  static_cast<unsigned>(shares));
  if (rt == 2) hipLaunchKernelGGL(lora_down_kernel<2>, grid, dim3(64 * kWaves), 0, stream, a);
  else hipLaunchKernelGGL(lora_down_kernel<1>, grid, dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace g355
