// The first factor of low-rank adapters: h[m] = scale[a] * (A[m] down_a), a = adapter[m].
//
// A workgroup has 16 rows, RT times 16 ranks and a share of K, of which its 8 waves
// take turns of 64 elements (a whole 128-byte line of every row). Rows and ranks are
// one v_mfma_f32_16x16x32_bf16's, read straight into its operands, eight turns of a wave
// in flight; every adapter that the 16 rows have is multiplied with its own rows. (A
// product's row depends on that row of A alone: nothing passes between requests.)
// The waves' sums are added in LDS in the order of the waves, the shares in theirs.
//
// Bound by the latency of its loads: a wave's are all in flight at once, a request to L2
// takes 500 to 1000 cycles, and the units that return data have some pending for 80% of
// the CUs' cycles. That a load touches 16 rows of 64 bytes (64 cache accesses, 16 if it
// took one row's 1024 bytes) is 13% of it: 12.0 us, 10.4 with loads of one row each, for
// 4096 rows, K = 4096, R = 16 and an adapter to every 16 rows. So only rows that have the
// adapter are read, and the reads are spread over the CUs: few rows have shares of K and
// adapters in workgroups of their own (a launch of more workgroups than that costs more than they
// bring: about 455 waves start in a microsecond). Measured: the same 4096 rows of six
// requests 16 us; 64 rows of 24 adapters, K = 14336, R = 64, 17 us (44 MB of adapters:
// 9 us at a copy's rate); one row 4 us.

#include "lora.hpp"

namespace g355 {

namespace {

constexpr int kWaves = 8;
constexpr int kTurn = 64;  // K elements of a wave's turn
constexpr int kMaxTiles = 1 << 20;

// The parts of one element (lora.hpp).
__device__ __forceinline__ void store_h(const LoraDownArgs& p, int m, int r, float h) {
  uint16_t* at = p.h + static_cast<int64_t>(m) * p.parts * p.pad + r;
  const auto store = [&](auto& part) {
    for (const uint32_t v : part) {
      *at = static_cast<uint16_t>(v);
      at += p.pad;
    }
  };
  if (p.parts == 3) {
    uint32_t part[3];
    split_h(h, part);
    store(part);
  } else {
    uint32_t part[2];
    split_h(h, part);
    store(part);
  }
}

}  // namespace

template <int RT>
__global__ void __launch_bounds__(64 * kWaves) lora_down_kernel(LoraDownArgs p) {
  constexpr int AHEAD = RT == 1 ? 8 : 4;  // turns whose loads are in flight
  __shared__ __attribute__((aligned(16))) float part[kWaves][RT][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane & 15, quarter = lane >> 4;
  const int r0 = blockIdx.y * 16 * RT;
  // Shares of one row tile are neighbours: rows are read as they lie in memory.
  const int parts = p.shares * p.split, part_of = blockIdx.x % parts;
  const int share = part_of % p.shares, first = part_of / p.shares, step = p.split;
  const int k_begin = share * p.share_len, k_end = min(p.K, k_begin + p.share_len);
  const int whole = (k_end - k_begin) / kTurn;  // turns without an end in them
  const int tiles = (p.M + 15) / 16;
  for (int tile = blockIdx.x / parts; tile < tiles; tile += gridDim.x / parts) {
    const int m = tile * 16 + l;
    int id = m < p.M ? p.adapter[m] : -1;
    id = id < p.adapters ? id : -1;
    unsigned left = static_cast<unsigned>(__ballot(id >= 0)) & 0xffffu;
    for (int turn = 0; left != 0; ++turn) {
      const int g = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
      const unsigned rows = static_cast<unsigned>(__ballot(id == g)) & 0xffffu;
      left &= ~rows;
      if (turn % step != first) continue;
      const float scale = p.scale ? p.scale[g] : 1.f;
      // Lanes of other rows read the adapter's first row along: the same lines.
      const uint16_t* x = p.A + (id == g ? m : tile * 16 + __builtin_ctz(rows)) * p.lda;

      const uint16_t* w[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t)
        w[t] = p.down + g * p.stride_down + min(r0 + 16 * t + l, p.rank - 1) * p.ld_down;
      f32x4 acc[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      // Whole turns, read without a look at the loaded values: AHEAD of them are
      // requested before the first is waited for.
      for (int t0 = wave; t0 < whole; t0 += kWaves * AHEAD) {
        i32x4 xv[AHEAD][2], wv[AHEAD][2][RT];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int t = t0 + u * kWaves;
          if (t >= whole) break;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int k = k_begin + t * kTurn + 32 * s + 8 * quarter;
            xv[u][s] = *reinterpret_cast<const i32x4_any*>(x + k);
#pragma unroll
            for (int q = 0; q < RT; ++q) wv[u][s][q] = *reinterpret_cast<const i32x4_any*>(w[q] + k);
          }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (t0 + u * kWaves >= whole) break;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int q = 0; q < RT; ++q)
              acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[u][s]),
                                                               __builtin_bit_cast(bf16x8, wv[u][s][q]), acc[q], 0, 0, 0);
        }
      }
      // The turn that K ends in.
      if (k_begin + whole * kTurn < k_end && wave == whole % kWaves) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int k = k_begin + whole * kTurn + 32 * s + 8 * quarter;
          const i32x4 xv = load8(x, k, p.K);
#pragma unroll
          for (int q = 0; q < RT; ++q)
            acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv),
                                                             __builtin_bit_cast(bf16x8, load8(w[q], k, p.K)), acc[q], 0, 0, 0);
        }
      }
      // Element e of lane l: row 4 (l / 16) + e, rank l % 16.
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][t][(4 * quarter + e) * 16 + l] = acc[t][e];
      __syncthreads();
      for (int q = tid; q < 256 * RT; q += 64 * kWaves) {
        const int t = q >> 8, i = q & 255, row = i >> 4, r = r0 + 16 * t + (i & 15);
        if (((rows >> row) & 1) && r < p.pad) {
          float h = part[0][t][i];
#pragma unroll
          for (int v = 1; v < kWaves; ++v) h += part[v][t][i];
          // Ranks past the last repeat it above, and are zeros in h.
          h = r < p.rank ? h * scale : 0.f;
          const int at = tile * 16 + row;
          if (p.h != nullptr && p.shares == 1) store_h(p, at, r, h);
          else p.partial[(static_cast<int64_t>(share) * p.M + at) * p.pad + r] = h;
        }
      }
      __syncthreads();
    }
  }
}

// The shares of K added up, in their order, for the tile kernels (adding them up
// there took 64 x 4096 x 14336 of rank 64 from 35 us to 45; this is 2).
__global__ void __launch_bounds__(256) lora_join_kernel(LoraDownArgs p) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.M * p.pad) return;
  const int m = i / p.pad, a = p.adapter[m];
  if (a < 0 || a >= p.adapters) return;
  float h = p.partial[i];
  for (int s = 1; s < p.shares; ++s) h += p.partial[static_cast<int64_t>(s) * p.M * p.pad + i];
  store_h(p, m, i - m * p.pad, h);
}

hipError_t launch_lora_down(const LoraDownArgs& a, hipStream_t stream) {
  const int tiles = (a.M + 15) / 16;
  // 32 ranks to a workgroup where the row tiles alone fill the card.
  const int rt = a.pad > 16 && tiles >= kLoraWorkgroups ? 2 : 1;
  const int x = tiles < kMaxTiles ? tiles : kMaxTiles, y = (a.pad + 16 * rt - 1) / (16 * rt);
  // Adapters of a tile go to workgroups of their own while there is room.
  LoraDownArgs d = a;
  const int64_t wgs = static_cast<int64_t>(x) * y * a.shares;
  d.split = static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, kLoraWorkgroups / wgs)));
  const dim3 grid(static_cast<unsigned>(x * a.shares * d.split), static_cast<unsigned>(y));
  if (rt == 2) hipLaunchKernelGGL(lora_down_kernel<2>, grid, dim3(64 * kWaves), 0, stream, d);
  else hipLaunchKernelGGL(lora_down_kernel<1>, grid, dim3(64 * kWaves), 0, stream, d);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.h == nullptr || a.shares == 1) return err;
  hipLaunchKernelGGL(lora_join_kernel, dim3(static_cast<unsigned>((a.M * a.pad + 255) / 256)), dim3(256), 0, stream, d);
  return hipGetLastError();
}

}  // namespace g355
