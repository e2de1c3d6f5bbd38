// Rows of tokens to their experts and back. The formulas are in gemm355.h.
//
// Everything here is bound by memory. Work is laid out by token, so that a
// token's own row (X, C or D) passes through HBM once, whatever top_k is, and
// the rows that experts read or wrote once each. A lane takes 8 elements (16
// bytes of BF16) at a time; its loads and stores need no alignment past the
// element's (gfx950 splits those that cross a line), so that odd widths and
// shifted rows run on the same kernels.

#include "common.hpp"
#include "routing.hpp"

namespace g355 {

namespace {

constexpr int kThreads = 256;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));

// Eight elements of a row as they lie in memory.
template <bool BF16>
struct Chunk {
  u32x4 v[BF16 ? 1 : 2];

  __device__ __forceinline__ float get(int q) const {
    if constexpr (BF16) {
      const uint32_t w = v[0][q >> 1];
      return __uint_as_float(q & 1 ? w & 0xffff0000u : w << 16);
    } else {
      return __uint_as_float(v[q >> 2][q & 3]);
    }
  }
};

// A lane's eight elements of a row, from element `at` on; those from lo up to hi
// are its own. The lane at the end of a row that is not a multiple of eight takes
// the row's last eight, of which the first belong to its neighbour; a row of fewer
// than eight has hi elements.
struct Span {
  int64_t at;
  int lo, hi;
};

__device__ __forceinline__ Span span_of(int64_t n, int N) {
  if (N < 8) return {0, 0, N};
  const int over = static_cast<int>(n) + 8 - N;
  return over > 0 ? Span{n - over, over, 8} : Span{n, 0, 8};
}

// NT: a row that is read once. (Non-temporal loads and stores of the rows on the
// experts' side, 8192 x 4 rows of 4096 there and back with gradients: 366 -> 330 us.)
template <bool BF16, bool NT>
__device__ __forceinline__ Chunk<BF16> load_chunk(const void* base, int64_t row, const Span& s) {
  Chunk<BF16> c;
  constexpr int ES = BF16 ? 2 : 4;
  const char* at = static_cast<const char*>(base) + (row + s.at) * ES;
  if (s.hi == 8) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
      const auto* from = reinterpret_cast<const u32x4_any*>(at + 16 * h);
      if constexpr (NT) c.v[h] = __builtin_nontemporal_load(from);
      else c.v[h] = *from;
    }
  } else {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) c.v[h] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int q = 0; q < 7; ++q) {
      if (q >= s.hi) continue;
      if constexpr (BF16)
        c.v[0][q >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[q]) << (16 * (q & 1));
      else
        c.v[q >> 2][q & 3] = reinterpret_cast<const uint32_t*>(at)[q];
    }
  }
  return c;
}

template <bool NT, class V>
__device__ __forceinline__ void store_any(void* at, const V& v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(at));
  else *reinterpret_cast<u32x4_any*>(at) = v;
}

template <bool BF16>
__device__ __forceinline__ void store_chunk(void* base, int64_t row, const Span& s, const float (&f)[8]) {
  constexpr int ES = BF16 ? 2 : 4;
  char* at = static_cast<char*>(base) + (row + s.at) * ES;
  uint32_t w[BF16 ? 4 : 8];
  if constexpr (BF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = f32x2_to_bf16x2_bits(f[2 * q], f[2 * q + 1]);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(f[q]);
  }
  if (s.lo == 0 && s.hi == 8) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h)
      store_any<true>(at + 16 * h, u32x4{w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]});
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q < s.lo || q >= s.hi) continue;
      if constexpr (BF16) reinterpret_cast<uint16_t*>(at)[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
      else reinterpret_cast<uint32_t*>(at)[q] = w[q];
    }
  }
}

// Threads along a row (a power of two) and rows of a workgroup, from the row's
// chunks: short rows share a workgroup.
struct RowGrid {
  int shift;
  dim3 grid;
};

RowGrid row_grid(int T, int64_t chunks) {
  RowGrid g;
  g.shift = 0;
  while (g.shift < 8 && (1 << g.shift) < chunks) ++g.shift;
  const int per = kThreads >> g.shift;
  const int64_t x = (static_cast<int64_t>(T) + per - 1) / per, y = (chunks + (1 << g.shift) - 1) >> g.shift;
  g.grid = dim3(static_cast<unsigned>(x < kMaxGrid ? x : kMaxGrid), static_cast<unsigned>(y < 1024 ? y : 1024));
  return g;
}

}  // namespace

// Rows of `nbytes` bytes, 16 to a lane. A row's last 16 bytes are taken as a
// whole, over the ones before them: the bytes that two lanes write are equal.
// BYTES: rows shorter than 16 bytes. NT: see launch_dispatch.
template <bool BYTES, bool NT>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(RowsArgs p, int64_t nbytes, int elem_bytes, int shift) {
  const int64_t ld_from = p.ld_from * elem_bytes, ld_to = p.ld_to * elem_bytes;
  const int sub = threadIdx.x & ((1 << shift) - 1), per = kThreads >> shift;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + (threadIdx.x >> shift); t < p.T;
       t += static_cast<int64_t>(gridDim.x) * per) {
    const int32_t* position = p.position + t * p.top_k;
    const char* from = static_cast<const char*>(p.from) + t * ld_from;
    char* to = static_cast<char*>(p.to);
    if constexpr (BYTES) {
      if (sub < nbytes) {
        const char v = from[sub];
        for (int j = 0; j < p.top_k; ++j) {
          const int r = position[j];
          if (r >= 0 && r < p.R) to[r * ld_to + sub] = v;
        }
      }
    } else {
      for (int64_t c = 16 * ((static_cast<int64_t>(blockIdx.y) << shift) + sub); c < nbytes;
           c += 16 * (static_cast<int64_t>(gridDim.y) << shift)) {
        const int64_t b = c + 16 <= nbytes ? c : nbytes - 16;
        const u32x4 v = *reinterpret_cast<const u32x4_any*>(from + b);
        for (int j = 0; j < p.top_k; ++j) {
          const int r = position[j];
          if (r >= 0 && r < p.R) store_any<NT>(to + r * ld_to + b, v);
        }
      }
    }
  }
}

// Four slots' rows are requested before the first is added: a lane has that many
// loads in flight.
template <bool YB, bool CB>
__global__ void __launch_bounds__(kThreads) combine_kernel(RowsArgs p, int shift) {
  constexpr int AHEAD = 4;
  const int sub = threadIdx.x & ((1 << shift) - 1), per = kThreads >> shift;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + (threadIdx.x >> shift); t < p.T;
       t += static_cast<int64_t>(gridDim.x) * per) {
    const int32_t* position = p.position + t * p.top_k;
    const float* weight = p.weight ? p.weight + t * p.top_k : nullptr;
    const int64_t row = t * p.ld_to;
    for (int64_t n = 8 * ((static_cast<int64_t>(blockIdx.y) << shift) + sub); n < p.N;
         n += 8 * (static_cast<int64_t>(gridDim.y) << shift)) {
      const Span span = span_of(n, p.N);
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j0 = 0; j0 < p.top_k; j0 += AHEAD) {
        Chunk<YB> y[AHEAD];
        float w[AHEAD];
        bool live[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const int j = j0 + a;
          const int r = j < p.top_k ? position[j] : -1;
          live[a] = r >= 0 && r < p.R;
          w[a] = weight && live[a] ? weight[j] : 1.f;
          if (live[a]) y[a] = load_chunk<YB, true>(p.from, r * p.ld_from, span);
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          if (!live[a]) continue;
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[a], y[a].get(q), acc[q]);
        }
      }
      if (p.beta != 0.f) {
        const Chunk<CB> c = load_chunk<CB, true>(p.to, row, span);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = fmaf(p.beta, c.get(q), acc[q]);
      }
      store_chunk<CB>(p.to, row, span, acc);
    }
  }
}

// W waves own a token (1 or 4). Four slots are taken at a time, so that D's row is
// read once for four of them and a lane has five loads in flight; a fifth slot
// reads it again, from cache. The waves' parts of a dot product are added in the
// order of the waves.
template <int W, bool DB, bool YB>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(RowsArgs p) {
  constexpr int AHEAD = 4;
  constexpr int TOKENS = kThreads / 64 / W;
  __shared__ float part[W > 1 ? kMaxSlots * W : 1];
  const int sub = threadIdx.x % (64 * W), lane = threadIdx.x & 63;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * TOKENS + threadIdx.x / (64 * W); t < p.T;
       t += static_cast<int64_t>(gridDim.x) * TOKENS) {
    for (int j0 = 0; j0 < p.top_k; j0 += AHEAD) {
      int r[AHEAD];
      float w[AHEAD], dot[AHEAD];
      bool any = false;
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int64_t s = t * p.top_k + j0 + a;
        r[a] = j0 + a < p.top_k ? p.position[s] : -1;
        r[a] = r[a] < p.R ? r[a] : -1;
        w[a] = p.weight && r[a] >= 0 ? p.weight[s] : 1.f;
        dot[a] = 0.f;
        any = any || r[a] >= 0;
      }
      if (any) {
        for (int64_t n = 8 * sub; n < p.N; n += 8 * 64 * W) {
          const Span span = span_of(n, p.N);
          Chunk<YB> y[AHEAD];
          if (p.dweight) {
#pragma unroll
            for (int a = 0; a < AHEAD; ++a)
              if (r[a] >= 0) y[a] = load_chunk<YB, true>(p.y, r[a] * p.ldy, span);
          }
          const Chunk<DB> d = load_chunk<DB, false>(p.from, t * p.ld_from, span);
#pragma unroll
          for (int a = 0; a < AHEAD; ++a) {
            if (r[a] < 0) continue;
            float f[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = w[a] * d.get(q);
            store_chunk<YB>(p.to, r[a] * p.ld_to, span, f);
            if (p.dweight) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (q >= span.lo && q < span.hi) dot[a] = fmaf(d.get(q), y[a].get(q), dot[a]);
            }
          }
        }
      }
      if (p.dweight) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          if (j0 + a >= p.top_k) break;
#pragma unroll
          for (int o = 32; o > 0; o >>= 1) dot[a] += __shfl_xor(dot[a], o);
          if constexpr (W == 1) {
            if (lane == 0) p.dweight[t * p.top_k + j0 + a] = dot[a];
          } else {
            if (lane == 0) part[W * (j0 + a) + (threadIdx.x >> 6)] = dot[a];
          }
        }
      }
    }
    if constexpr (W > 1) {
      if (p.dweight) {
        __syncthreads();
        if (sub < p.top_k) {
          float dot = part[W * sub];
#pragma unroll
          for (int w = 1; w < W; ++w) dot += part[W * sub + w];
          p.dweight[t * p.top_k + sub] = dot;
        }
        __syncthreads();  // the next token's parts come after
      }
    }
  }
}

hipError_t launch_dispatch(const RowsArgs& a, int elem_bytes, hipStream_t stream) {
  const int64_t nbytes = static_cast<int64_t>(a.N) * elem_bytes;
  const RowGrid g = row_grid(a.T, nbytes < 16 ? 16 : (nbytes + 15) / 16);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, g.grid, dim3(kThreads), 0, stream, a, nbytes, elem_bytes, g.shift);
  };
  // Rows that the memory-side cache (256 MB) cannot keep for their reader are
  // stored non-temporally (268 MB of them: 2% less of a pass there and back);
  // others are not (a pass over 25 MB: 58.1 us, with them 59.5).
  if (nbytes < 16) go(dispatch_kernel<true, false>);
  else if (nbytes * a.top_k * a.T >= int64_t{256} << 20) go(dispatch_kernel<false, true>);
  else go(dispatch_kernel<false, false>);
  return hipGetLastError();
}

hipError_t launch_combine(const RowsArgs& a, bool y_bf16, bool c_bf16, hipStream_t stream) {
  const RowGrid g = row_grid(a.T, (static_cast<int64_t>(a.N) + 7) / 8);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, g.grid, dim3(kThreads), 0, stream, a, g.shift); };
  if (y_bf16) c_bf16 ? go(combine_kernel<true, true>) : go(combine_kernel<true, false>);
  else c_bf16 ? go(combine_kernel<false, true>) : go(combine_kernel<false, false>);
  return hipGetLastError();
}

template <int W>
static hipError_t launch_combine_grad_w(const RowsArgs& a, bool d_bf16, bool y_bf16, hipStream_t stream) {
  constexpr int TOKENS = kThreads / 64 / W;
  const int wgs = (a.T + TOKENS - 1) / TOKENS;
  const dim3 grid(static_cast<unsigned>(wgs < kMaxGrid ? wgs : kMaxGrid));
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a); };
  if (d_bf16) y_bf16 ? go(combine_grad_kernel<W, true, true>) : go(combine_grad_kernel<W, true, false>);
  else y_bf16 ? go(combine_grad_kernel<W, false, true>) : go(combine_grad_kernel<W, false, false>);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const RowsArgs& a, bool d_bf16, bool y_bf16, hipStream_t stream) {
  // A wave per token where it covers the row in one or two steps.
  return a.N > 1024 ? launch_combine_grad_w<4>(a, d_bf16, y_bf16, stream)
                    : launch_combine_grad_w<1>(a, d_bf16, y_bf16, stream);
}

}  // namespace g355
