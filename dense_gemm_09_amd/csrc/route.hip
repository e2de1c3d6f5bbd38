// Routing of tokens to experts, its gradient, and the order of rows by expert.
// The formulas are in gemm355.h.

#include "common.hpp"
#include "routing.hpp"

namespace g355 {

namespace {

constexpr int kThreads = 256;  // four waves, a token each

__device__ __forceinline__ float load_logit(const void* p, int64_t i, bool bf16) {
  return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <class V>
__device__ __forceinline__ V wave_top(V v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const V u = __shfl_xor(v, o);
    v = u > v ? u : v;
  }
  return v;
}

// The largest value of a wave's lanes and the lowest index that has it.
__device__ __forceinline__ void wave_best(double& v, int& at) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const double u = __shfl_xor(v, o);
    const int b = __shfl_xor(at, o);
    if (u > v || (u == v && b < at)) {
      v = u;
      at = b;
    }
  }
}

// log of the logistic function, without overflow on either side.
__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.f) - log1pf(expf(-fabsf(x))); }

}  // namespace

// ------------------------------------------------------------------ choice

// One wave per token; lane l holds experts l, l + 64, ... (EPL of them).
template <int EPL>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteArgs p, bool bf16) {
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_inff();
  for (int t = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); t < p.T; t += gridDim.x * (kThreads / 64)) {

  float x[EPL];
  bool bad = false;
  float top = ninf;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.E ? load_logit(p.logits, t * p.ldl + e, bf16) : ninf;
    bad = bad || x[i] != x[i] || (!p.sigmoid && x[i] == -ninf);
    top = fmaxf(top, x[i]);
  }
  int32_t* expert = p.expert + static_cast<int64_t>(t) * p.top_k;
  float* weight = p.weight + static_cast<int64_t>(t) * p.top_k;
  if (__any(bad)) {
    if (lane < p.top_k) {
      expert[lane] = -1;
      weight[lane] = __builtin_nanf("");
    }
    continue;
  }
  top = wave_top(top);
  const float base = p.sigmoid || top == ninf ? 0.f : top;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) sum += expf(x[i] - base);
  sum = wave_sum(sum);

  // Scores to choose by, in 64 bits: experts whose scores differ in their last
  // bits are told apart. Without a bias they are the logits.
  const bool by_logit = p.bias == nullptr && p.group_best == 1;
  double c[EPL];
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = x[i];
  } else {
    double all = 1.0;
    if (!p.sigmoid) {
      all = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) all += exp(static_cast<double>(x[i]) - base);
      all = wave_sum(all);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      const double xd = x[i];
      double v = p.sigmoid ? 1.0 / (1.0 + exp(-xd)) : exp(xd - base) / all;
      if (p.bias != nullptr && e < p.E) v += p.bias[e];
      c[i] = x[i] > ninf && v == v ? v : ninf;
    }
  }

  if (p.groups > 1) {
    const int per = p.E / p.groups;
    double mine = ninf;  // score of group `lane`
    for (int g = 0; g < p.groups; ++g) {
      double total = ninf;
      int first = -1;
      for (int b = 0; b < p.group_best; ++b) {
        double v = ninf;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane + 64 * i;
          if (e / per == g && e < p.E && e != first && c[i] > v) {
            v = c[i];
            at = e;
          }
        }
        wave_best(v, at);
        if (v > ninf) total = b == 0 ? v : total + v;
        first = at;
      }
      if (lane == g) mine = total;
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double v = __shfl(mine, g);
      if (v > mine || (v == mine && g < lane)) ++rank;
    }
    const unsigned long long keep = __ballot(lane < p.groups && rank < p.top_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < p.E && !((keep >> (e / per)) & 1)) c[i] = ninf;
    }
  }

  int id = -1;  // lane j: the j-th expert and its logit
  float xj = ninf;
  for (int j = 0; j < p.top_k; ++j) {
    double v = ninf;
    int at = 1 << 30;
    float xv = ninf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (c[i] > v) {
        v = c[i];
        at = lane + 64 * i;
        xv = x[i];
      }
    }
    wave_best(v, at);
    if (!(v > ninf)) break;
    xv = __shfl(xv, at & 63);
    if (lane == j) {
      id = at;
      xj = xv;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 64 * i == at) c[i] = ninf;
  }

  float w = 0.f;
  if (p.renormalise) {
    const float ls = p.sigmoid ? log_sigmoid(xj) : xj;
    const float most = wave_top(id >= 0 ? ls : ninf);
    const float s = id >= 0 ? expf(ls - most) : 0.f;
    const float z = wave_sum(s);
    w = id >= 0 ? p.scale * (s / z) : 0.f;
  } else if (id >= 0) {
    w = p.scale * (p.sigmoid ? expf(log_sigmoid(xj)) : expf(xj - base) / sum);
  }
  if (lane < p.top_k) {
    expert[lane] = id;
    weight[lane] = w;
  }
  }
}

// ---------------------------------------------------------------- gradient

// One wave per token; lane j has slot j while the slots' gradients are formed.
template <int EPL>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(RouteGradArgs p, bool bf16) {
  const int lane = threadIdx.x & 63;
  for (int t = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); t < p.T; t += gridDim.x * (kThreads / 64)) {
  const float ninf = -__builtin_inff();
  const bool full = !p.sigmoid && !p.renormalise;  // every logit has a gradient

  int id = -1;
  float dw = 0.f, xj = ninf;
  if (lane < p.top_k) {
    id = p.expert[static_cast<int64_t>(t) * p.top_k + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      dw = p.scale * p.dweight[static_cast<int64_t>(t) * p.top_k + lane];
      xj = load_logit(p.logits, t * p.ldl + id, bf16);
    }
  }

  float x[EPL], base = 0.f, sum = 1.f;
  if (full) {
    float top = ninf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      x[i] = e < p.E ? load_logit(p.logits, t * p.ldl + e, bf16) : ninf;
      top = fmaxf(top, x[i]);
    }
    top = wave_top(top);
    base = top == ninf ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += expf(x[i] - base);
    sum = wave_sum(sum);
  }

  float v = 0.f, dot = 0.f;
  if (p.renormalise) {
    const float ls = p.sigmoid ? log_sigmoid(xj) : xj;
    const float most = wave_top(id >= 0 ? ls : ninf);
    const float s = id >= 0 && most > ninf ? expf(ls - most) : 0.f;
    const float z = wave_sum(s);
    const float share = s > 0.f ? s / z : 0.f;
    const float mean = wave_sum(id >= 0 ? dw * share : 0.f);
    v = id >= 0 ? share * (dw - mean) : 0.f;
    if (p.sigmoid && id >= 0) v *= 1.f / (1.f + expf(xj));
  } else if (p.sigmoid) {
    // s (1 - s), both factors to their relative accuracy
    if (id >= 0) v = dw * expf(log_sigmoid(xj)) * (1.f / (1.f + expf(xj)));
  } else {
    v = id >= 0 ? dw * (expf(xj - base) / sum) : 0.f;
    dot = wave_sum(v);
  }
  const bool none = !__any(id >= 0);

  float d[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) d[i] = full && !none ? -dot * (expf(x[i] - base) / sum) : 0.f;
  for (int j = 0; j < p.top_k; ++j) {
    const int at = __shfl(id, j);
    const float add = __shfl(v, j);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 64 * i == at) d[i] += add;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    if (bf16) static_cast<uint16_t*>(p.dlogits)[t * p.ldd + e] = f32_to_bf16_bits(d[i]);
    else static_cast<float*>(p.dlogits)[t * p.ldd + e] = d[i];
  }
  }
}

template <class Args, class F>
static hipError_t launch_rows_of_experts(const Args& a, bool bf16, F kernel_of, hipStream_t stream) {
  const int wgs = (a.T + kThreads / 64 - 1) / (kThreads / 64);
  const dim3 grid(static_cast<unsigned>(wgs < kMaxGrid ? wgs : kMaxGrid)), block(kThreads);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, bf16); };
  kernel_of(go);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  return launch_rows_of_experts(a, bf16, [&](auto go) {
    if (a.E <= 64) go(route_kernel<1>);
    else if (a.E <= 256) go(route_kernel<4>);
    else go(route_kernel<16>);
  }, stream);
}

hipError_t launch_route_grad(const RouteGradArgs& a, bool bf16, hipStream_t stream) {
  return launch_rows_of_experts(a, bf16, [&](auto go) {
    if (a.E <= 64) go(route_grad_kernel<1>);
    else if (a.E <= 256) go(route_grad_kernel<4>);
    else go(route_grad_kernel<16>);
  }, stream);
}

// ------------------------------------------------------------- order of rows

// A stable counting sort. Slots are divided into chunks, chunks into a segment
// for each wave of a workgroup. Up to kSmallSlots slots are one chunk and one
// launch; otherwise a first launch counts every chunk's experts, and in the
// second every workgroup adds up the counts of the chunks (there are at most
// kMaxChunks), which gives the first row of each expert in its chunk, and places
// its slots. Slots without an expert are an expert G behind the others. Within a
// wave, slots of one expert find each other by ballots over the expert's bits, 64
// at a time. The only atomics add up integers: no result depends on their order.
//
// All of it is latency: a second launch costs more than what it does (32768 slots of 64
// experts: three launches with a scan of their own took 15 us).

constexpr int kSmallWaves = 16;      // 512 slots a wave, eight to a lane
constexpr int kOrderWaves = 4;
constexpr int kHeldKeys = 8;         // keys that a lane holds at a time
constexpr int kMaxChunks = 128;

__device__ __forceinline__ int expert_key(const OrderArgs& p, int s) {
  const int e = p.expert[s];
  return e >= 0 && e < p.G ? e : p.G;
}

// Keys of slots s0 + 64 h + lane below `end` (-1 past it).
__device__ __forceinline__ void load_keys(const OrderArgs& p, int s0, int end, int lane, int (&key)[kHeldKeys]) {
#pragma unroll
  for (int h = 0; h < kHeldKeys; ++h) {
    const int s = s0 + 64 * h + lane;
    key[h] = s < end ? expert_key(p, s) : -1;
  }
}

// Counts the experts of slots [begin, end) in a wave's counters.
__device__ __forceinline__ void count_keys(const OrderArgs& p, int begin, int end, int lane, int* counter) {
  for (int s0 = begin; s0 < end; s0 += 64 * kHeldKeys) {
    int key[kHeldKeys];
    load_keys(p, s0, end, lane, key);
#pragma unroll
    for (int h = 0; h < kHeldKeys; ++h)
      if (key[h] >= 0) atomicAdd(&counter[key[h]], 1);
  }
}

// LDS of this wave as its other lanes have left it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__global__ void __launch_bounds__(64 * kOrderWaves) order_count_kernel(OrderArgs p) {
  extern __shared__ int counter[];
  for (int g = threadIdx.x; g <= p.G; g += 64 * kOrderWaves) counter[g] = 0;
  __syncthreads();
  const int begin = blockIdx.x * p.chunk, end = min(p.S, begin + p.chunk);
  const int seg = p.chunk / kOrderWaves;  // a multiple of 64
  const int wave = threadIdx.x >> 6, from = begin + wave * seg;
  count_keys(p, from, min(end, from + seg), threadIdx.x & 63, counter);
  __syncthreads();
  int32_t* out = p.counts + static_cast<int64_t>(blockIdx.x) * (p.G + 1);
  for (int g = threadIdx.x; g <= p.G; g += 64 * kOrderWaves) out[g] = counter[g];
}

// WAVES counters of G + 1 experts in LDS. SMALL: the only workgroup.
template <int WAVES, bool SMALL>
__global__ void __launch_bounds__(64 * WAVES) order_place_kernel(OrderArgs p) {
  extern __shared__ int counter[];
  __shared__ int part[WAVES];
  constexpr int NT = 64 * WAVES;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bins = p.G + 1;
  const int chunk = static_cast<int>(blockIdx.x);
  const int begin = chunk * p.chunk, end = min(p.S, begin + p.chunk);
  const int seg = p.chunk / WAVES;
  const int from = begin + wave * seg, to = min(end, from + seg);

  for (int i = tid; i < WAVES * bins; i += NT) counter[i] = 0;
  __syncthreads();
  int* mine = counter + wave * bins;
  count_keys(p, from, to, lane, mine);
  __syncthreads();

  // Counters become first rows: of the experts in order, in each the chunks
  // before this one, in that the waves.
  int carry = 0;  // rows of the experts before this round's
  for (int g0 = 0; g0 < bins; g0 += NT) {
    const int g = g0 + tid;
    int total = 0, before = 0;
    if (g < bins) {
      if constexpr (SMALL) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) total += counter[w * bins + g];
      } else {
#pragma unroll 8
        for (int c = 0; c < p.chunks; ++c) {
          const int n = p.counts[static_cast<int64_t>(c) * bins + g];
          total += n;
          before += c < chunk ? n : 0;
        }
      }
    }
    int incl = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      incl += lane >= o ? v : 0;
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int row = carry + incl - total;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      row += w < wave ? part[w] : 0;
      carry += part[w];
    }
    if (g < bins) {
      if (chunk == 0) p.offsets[g] = row;
      row += before;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int n = counter[w * bins + g];
        counter[w * bins + g] = row;
        row += n;
      }
    }
    __syncthreads();
  }

  int bits = 0;
  while ((p.G >> bits) != 0) ++bits;
  for (int s0 = from; s0 < to; s0 += 64 * kHeldKeys) {
    int key[kHeldKeys];
    load_keys(p, s0, to, lane, key);
#pragma unroll
    for (int h = 0; h < kHeldKeys; ++h) {
      const int s = s0 + 64 * h + lane;
      const bool in_range = key[h] >= 0;
      unsigned long long same = __ballot(in_range);  // lanes with the same expert
      if (same == 0) break;
      for (int b = 0; b < bits; ++b) {
        const bool set = (key[h] >> b) & 1;
        const unsigned long long with = __ballot(set);
        same &= set ? with : ~with;
      }
      int first = 0;
      if (in_range) first = mine[key[h]];
      wave_fence();
      if (in_range) {
        // The last of them moves the counter on.
        if ((same >> lane) == 1) mine[key[h]] = first + __popcll(same);
        const int row = first + __popcll(same & ((1ull << lane) - 1));
        const bool live = key[h] < p.G;
        p.position[s] = live ? row : -1;
        if (p.order) p.order[row] = live ? s : -1;
      }
      wave_fence();
    }
  }
}

void order_chunks(int64_t S, int64_t G, int& chunk, int& chunks) {
  if (order_small(S, G)) {
    chunk = static_cast<int>((S + 64 * kSmallWaves - 1) / (64 * kSmallWaves) * (64 * kSmallWaves));
    chunks = 1;
    return;
  }
  const int64_t least = 64 * kHeldKeys * kOrderWaves, per = (S + kMaxChunks - 1) / kMaxChunks;
  chunk = static_cast<int>((per + least - 1) / least * least);
  chunks = static_cast<int>((S + chunk - 1) / chunk);
}

hipError_t launch_order(const OrderArgs& a, hipStream_t stream) {
  const size_t lds = static_cast<size_t>(a.G + 1) * sizeof(int);
  if (order_small(a.S, a.G)) {
    hipLaunchKernelGGL((order_place_kernel<kSmallWaves, true>), dim3(1), dim3(64 * kSmallWaves), kSmallWaves * lds,
                       stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(order_count_kernel, dim3(a.chunks), dim3(64 * kOrderWaves), lds, stream, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((order_place_kernel<kOrderWaves, false>), dim3(a.chunks), dim3(64 * kOrderWaves),
                     kOrderWaves * lds, stream, a);
  return hipGetLastError();
}

}  // namespace g355
