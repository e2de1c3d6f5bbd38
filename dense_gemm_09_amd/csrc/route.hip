// Routing of tokens to experts, its gradient, and the order of rows by expert.
// The formulas are in gemm355.h.

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "routing.hpp"

namespace g355 {

namespace {

constexpr int kThreads = 256;  // four waves, a token each

typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// Lane l's experts l * EPL .. l * EPL + EPL - 1 of the row at element `row`; -inf past E.
template <int EPL, bool BF16>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int E, int lane, float (&x)[EPL]) {
  const int e0 = lane * EPL;
  constexpr int BYTES = EPL * (BF16 ? 2 : 4);
  if (BYTES >= 8 && e0 + EPL <= E) {
    const char* at = static_cast<const char*>(p) + (row + e0) * (BF16 ? 2 : 4);
    uint32_t w[BYTES >= 8 ? BYTES / 4 : 2];
    if constexpr (BYTES == 8) {
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(at);
      w[0] = v[0];
      w[1] = v[1];
    } else if constexpr (BYTES > 8) {
#pragma unroll
      for (int h = 0; h < BYTES / 16; ++h) {
        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(at + 16 * h);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[4 * h + q] = v[q];
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (BF16) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else x[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = e0 + i < E ? load_logit<BF16>(p, row + e0 + i) : -__builtin_inff();
  }
}

// The value of a wave's last lane after a scan along it that combines neighbours.
// (Shifts by 1, 2, 4 and 8 lanes within rows of 16, then the rows' last lanes
// carried over.) Lanes that a shift leaves without a neighbour combine with `idle`.
template <class F>
__device__ __forceinline__ int wave_fold(int v, int idle, F combine) {
  v = combine(v, __builtin_amdgcn_update_dpp(idle, v, 0x111, 0xf, 0xf, false));
  v = combine(v, __builtin_amdgcn_update_dpp(idle, v, 0x112, 0xf, 0xf, false));
  v = combine(v, __builtin_amdgcn_update_dpp(idle, v, 0x114, 0xf, 0xf, false));
  v = combine(v, __builtin_amdgcn_update_dpp(idle, v, 0x118, 0xf, 0xf, false));
  v = combine(v, __builtin_amdgcn_update_dpp(idle, v, 0x142, 0xa, 0xf, false));
  v = combine(v, __builtin_amdgcn_update_dpp(idle, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(wave_fold(__float_as_int(v), 0, [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

__device__ __forceinline__ int wave_max(int v) {
  return wave_fold(v, INT32_MIN, [](int a, int b) { return max(a, b); });
}

// The same for doubles.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double idle, double v) {
  const uint64_t a = __builtin_bit_cast(uint64_t, idle), b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(static_cast<int>(a), static_cast<int>(b), CTRL, ROWS, 0xf, false);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(static_cast<int>(a >> 32), static_cast<int>(b >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double lane_f64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

template <class F>
__device__ __forceinline__ double wave_fold(double v, double idle, F combine) {
  v = combine(v, dpp_f64<0x111, 0xf>(idle, v));
  v = combine(v, dpp_f64<0x112, 0xf>(idle, v));
  v = combine(v, dpp_f64<0x114, 0xf>(idle, v));
  v = combine(v, dpp_f64<0x118, 0xf>(idle, v));
  v = combine(v, dpp_f64<0x142, 0xa>(idle, v));
  v = combine(v, dpp_f64<0x143, 0xc>(idle, v));
  return lane_f64(v, 63);
}

__device__ __forceinline__ double wave_sum(double v) {
  return wave_fold(v, 0.0, [](double a, double b) { return a + b; });
}

__device__ __forceinline__ double wave_max(double v) {
  return wave_fold(v, -__builtin_inf(), [](double a, double b) { return a > b ? a : b; });
}

// Floats as integers in the same order (-0 below +0: the callers add 0 first),
// whose maximum needs one instruction. Its own inverse.
__device__ __forceinline__ int order_key(int bits) { return bits ^ ((bits >> 31) & 0x7fffffff); }
__device__ __forceinline__ int key_of(float v) { return order_key(__float_as_int(v + 0.f)); }
__device__ __forceinline__ float value_of(int key) { return __int_as_float(order_key(key)); }
constexpr int kNoKey = static_cast<int>(0x807fffffu);  // key_of(-inf)

__device__ __forceinline__ float wave_top(float v) { return value_of(wave_max(key_of(v))); }

// Keys to choose by: integers in the order of FP32 values, or 64-bit scores.
template <class Key>
struct KeyOf;
template <>
struct KeyOf<int> {
  using Score = float;
  __device__ static constexpr int none() { return kNoKey; }
  __device__ __forceinline__ static float score(int k) { return value_of(k); }
  __device__ __forceinline__ static float lane(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
  }
};
template <>
struct KeyOf<double> {
  using Score = double;
  __device__ static constexpr double none() { return -__builtin_inf(); }
  __device__ __forceinline__ static double score(double k) { return k; }
  __device__ __forceinline__ static double lane(double v, int l) { return lane_f64(v, l); }
};

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// log of the logistic function, without overflow on either side.
__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.f) - log1pf(expf(-fabsf(x))); }

// exp(a - b), with what the rounding of the difference drops: up to 2^-24 of it, which
// the exponential would turn into an error that grows with the distance (of a logit 80
// below the largest: 64 last bits). Finite a and b, or an a of -inf.
__device__ __forceinline__ float exp_difference(float a, float b) {
  const float d = a - b, s = d - a;
  const float dropped = (a - (d - s)) - (b + s);
  return expf(d) * (d > -__FLT_MAX__ ? 1.f + dropped : 1.f);
}

}  // namespace

// ------------------------------------------------------------------ choice
//
// One wave per token; a lane has EPL neighbouring experts. Everything a choice
// needs of the whole row is a wave's scan (six instructions) and scalar from
// there on: the best key is found with a maximum, its expert from the lanes' equality
// masks, lowest lane and lowest element first, in scalar registers. With E = 256
// a round is one chain of about 40 vector and scalar instructions.
//
// Without a bias the keys are the logits. With one, scores are first formed in
// FP32, each within `slack` of its exact value; where two neighbours in the order
// found (or the last group kept and the first not) are closer than that decides,
// the token is done again with scores in 64 bits. With 256 experts, random logits
// and a bias that happens to one token in 700 (16384 tokens: 64-bit scores for all
// of them 98 us, this 27).

// The lane `step` away within 16 lanes, for butterflies: pairs, quads, and then
// mirrored halves, whose lanes agree by then.
template <int STEP>
constexpr int kAcross = STEP == 1 ? 0xb1 : STEP == 2 ? 0x4e : STEP == 4 ? 0x141 : 0x140;
template <int STEP>
__device__ __forceinline__ int across(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kAcross<STEP>, 0xf, 0xf, true);
}
template <int STEP>
__device__ __forceinline__ double across(double v) {
  return dpp_f64<kAcross<STEP>, 0xf>(v, v);
}

template <class V>
__device__ __forceinline__ V larger(V a, V b) { return a > b ? a : b; }
template <class V>
__device__ __forceinline__ V smaller(V a, V b) { return a > b ? b : a; }

template <class K, class Key>
__device__ __forceinline__ typename K::Score group_total(const RouteArgs& p, Key best, Key second) {
  using Score = typename K::Score;
  if (p.group_best == 1) return K::score(best);
  const Score half = Score(0.5) * K::score(best);
  return second != K::none() ? half + Score(0.5) * K::score(second) : half;
}

// The scores of the groups, group g's in lane g: its best key, or half the sum of its two
// best (the sum itself may be beyond FP32 where biases are large). In the usual case a group is 1, 2, 4, 8 or 16 lanes whole, which find its two
// best in a butterfly, all groups at once; otherwise it is one group after another.
template <int EPL, class Key>
__device__ __forceinline__ typename KeyOf<Key>::Score group_scores(const RouteArgs& p, const Key (&key)[EPL], int lane) {
  using K = KeyOf<Key>;
  using Score = typename K::Score;
  constexpr Key none = K::none();
  const int per = p.E / p.groups, lanes = per / EPL;
  Score mine = -__builtin_inff();
  if (lanes * EPL == per && (lanes & (lanes - 1)) == 0 && lanes >= 1 && lanes <= 16) {
    Key a = none, b = none;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      b = larger(b, smaller(a, key[i]));
      a = larger(a, key[i]);
    }
    const auto join = [&](Key a2, Key b2) {
      b = larger(larger(b, b2), smaller(a, a2));
      a = larger(a, a2);
    };
    if (lanes > 1) join(across<1>(a), across<1>(b));
    if (lanes > 2) join(across<2>(a), across<2>(b));
    if (lanes > 4) join(across<4>(a), across<4>(b));
    if (lanes > 8) join(across<8>(a), across<8>(b));
    const Score total = group_total<K>(p, a, b);
    const Score there = __shfl(total, (lane * lanes) & 63);
    return lane < p.groups ? there : mine;
  }
  for (int g = 0; g < p.groups; ++g) {
    Key a = none, b = none;
    const int lo = g * per - lane * EPL, hi = lo + per;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const Key k = i >= lo && i < hi ? key[i] : none;
      b = larger(b, smaller(a, k));
      a = larger(a, k);
    }
    const Key best = wave_max(a);
    Key second = none;
    if (p.group_best == 2 && best != none) {
      const int owner = __builtin_ctzll(__ballot(a == best));
      second = wave_max(lane == owner ? b : a);
    }
    const Score total = group_total<K>(p, best, second);
    if (lane == g) mine = total;
  }
  return mine;
}

// Removes the experts outside the best groups from `key`. Returns whether
// slack leaves the groups in doubt.
template <int EPL, class Key>
__device__ __forceinline__ bool keep_groups(const RouteArgs& p, Key (&key)[EPL], int lane, float slack) {
  using K = KeyOf<Key>;
  const int per = p.E / p.groups;
  const auto mine = group_scores<EPL, Key>(p, key, lane);
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const auto v = K::lane(mine, g);
    rank += (v > mine) | ((v == mine) & (g < lane)) ? 1 : 0;
  }
  const bool kept = lane < p.groups && rank < p.top_groups;
  const unsigned long long keep = __ballot(kept);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    key[i] = (keep >> ((e / per) & 63)) & 1 ? key[i] : K::none();  // (past E there is none anyway)
  }
  if (slack == 0.f || p.top_groups == p.groups) return false;
  const float last = -wave_top(kept ? -static_cast<float>(mine) : -__builtin_inff());
  const float next = wave_top(kept ? -__builtin_inff() : static_cast<float>(mine));
  // (Groups without an expert left are -inf on both sides: inf - inf is NaN, no doubt.)
  return last - next <= 2.f * slack;
}

// Rounds: slot j's expert goes to lane j's id (-1: none left). With a slack, one round
// more tells how near the first expert left out is; returns whether the order is in doubt.
template <int EPL, class Key>
__device__ __forceinline__ bool choose(const RouteArgs& p, Key (&key)[EPL], int lane, float slack, int& id) {
  using K = KeyOf<Key>;
  bool doubt = false;
  auto before = K::score(K::none());
  before = -before;
  const int rounds = slack > 0.f ? p.top_k + 1 : p.top_k;
  id = -1;
  for (int j = 0; j < rounds; ++j) {
    Key v = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) v = larger(v, key[i]);
    const Key best = wave_max(v);
    if (best == K::none()) break;
    const int owner = __builtin_ctzll(__ballot(v == best));
    // The lowest element of the owner's that has it.
    int at = EPL - 1;
#pragma unroll
    for (int i = EPL - 2; i >= 0; --i)
      if ((__ballot(key[i] == best) >> owner) & 1) at = i;
    if (slack > 0.f) {
      const auto here = K::score(best);
      doubt |= before - here <= 2.f * slack;
      before = here;
    }
    id = lane == j ? owner * EPL + at : id;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = (lane == owner) & (i == at) ? K::none() : key[i];
  }
  if (lane >= p.top_k) id = -1;
  return doubt;
}

// One token's choice with scores in 64 bits.
template <int EPL>
__device__ __forceinline__ void choose_exactly(const RouteArgs& p, const float (&x)[EPL], const float (&bias)[EPL],
                                               float base, int lane, int& id) {
  const double ninf = -__builtin_inf();
  double c[EPL], all = 1.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const double xd = x[i];
    c[i] = exp(p.sigmoid ? -xd : xd - base);
  }
  if (!p.sigmoid) {
    all = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) all += c[i];
    all = wave_sum(all);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const double v = (p.sigmoid ? 1.0 / (1.0 + c[i]) : c[i] / all) + bias[i];
    c[i] = x[i] > -__builtin_inff() && v == v ? v : ninf;
  }
  if (p.groups > 1) keep_groups<EPL, double>(p, c, lane, 0.f);
  choose<EPL, double>(p, c, lane, 0.f, id);
}

// SCORED: keys are scores (a bias, or groups by two scores), not logits. Up to 256
// experts, six waves to a SIMD: the 64-bit scores, rarely needed, would take the
// registers of one (16384 tokens of 256 experts with gradient: 35.4 us, so 32.5).
template <int EPL, bool BF16, bool SCORED>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(EPL <= 4 ? 6 : 1))) route_kernel(RouteArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float ninf = -__builtin_inff();
  const float most_allowed = p.sigmoid ? __builtin_inff() : __FLT_MAX__;
  const int step = gridDim.x * (kThreads / 64);
  int t = blockIdx.x * (kThreads / 64) + wave;
  if (t >= p.T) return;

  float bias[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) bias[i] = 0.f;
  if constexpr (SCORED) {
    if (p.bias != nullptr) load_row<EPL, false>(p.bias, 0, p.E, lane, bias);  // (past E -inf: no key)
  }
  float x[EPL];
  load_row<EPL, BF16>(p.logits, t * p.ldl, p.E, lane, x);
  for (;;) {
    int32_t* expert = p.expert + static_cast<int64_t>(t) * p.top_k;
    float* weight = p.weight + static_cast<int64_t>(t) * p.top_k;
    // The next token's logits are on their way while this one's are sorted out.
    t += step;
    const bool more = t < p.T;
    float next[EPL];
    if (more) load_row<EPL, BF16>(p.logits, t * p.ldl, p.E, lane, next);

    float top = ninf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      bad |= !(x[i] <= most_allowed);
      top = x[i] > top ? x[i] : top;
    }
    int id = -1;
    float w = 0.f;
    if (__any(bad)) {
      w = __builtin_nanf("");
    } else {
      // Softmax: the row's largest logit and the sum. Both scores and weights as
      // they are need it, shares of the chosen do not.
      float base = 0.f, sum = 1.f;
      if (!p.sigmoid && (SCORED || !p.renormalise)) {
        top = wave_top(top);
        base = top == ninf ? 0.f : top;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sum += fast_exp(x[i] - base);
        sum = wave_sum(sum);
      }

      int key[EPL];
      float slack = 0.f;
      if constexpr (!SCORED) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = key_of(x[i]);
      } else {
        // How far a c may be off: the exponential of an argument off by 2^-24 of itself and
        // one more step of 2^-23, the reciprocal's, and half a step of the sum with
        // the bias. A sigmoid, at most 1, comes to 2^-22; a softmax's, at most 1 / sum,
        // to 2^-22 of that and the 22 roundings of the sum.
        float most = 0.f;
        const float inverse = 1.f / sum;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const float s = p.sigmoid ? __builtin_amdgcn_rcpf(1.f + fast_exp(-x[i])) : fast_exp(x[i] - base) * inverse;
          const float c = s + bias[i];
          const bool there = (x[i] > ninf) & (c > ninf);  // (false for a NaN)
          key[i] = there ? key_of(c) : kNoKey;
          most = there & (fabsf(c) > most) ? fabsf(c) : most;
        }
        slack = (p.sigmoid ? 0x1p-20f : 0x1p-19f * inverse) + 0x1p-22f * wave_top(most);
      }
      bool doubt = false;
      if (p.groups > 1) doubt = keep_groups<EPL, int>(p, key, lane, slack);
      doubt |= choose<EPL, int>(p, key, lane, slack, id);
      if constexpr (SCORED) {
        if (__any(doubt)) choose_exactly<EPL>(p, x, bias, base, lane, id);
      }

      float xj = ninf;  // its logit, from the lane that has it
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float u = __shfl(x[i], (id >= 0 ? id : 0) / EPL);
        xj = (id >= 0) & (id % EPL == i) ? u : xj;
      }
      if (p.renormalise) {
        const float ls = p.sigmoid ? log_sigmoid(xj) : xj;
        const float most = wave_top(id >= 0 ? ls : ninf);
        const float s = id >= 0 ? exp_difference(ls, most) : 0.f;
        const float z = wave_sum(s);
        w = id >= 0 ? p.scale * (s / z) : 0.f;
      } else if (id >= 0) {
        w = p.scale * (p.sigmoid ? expf(log_sigmoid(xj)) : exp_difference(xj, base) / sum);
      }
    }
    if (lane < p.top_k) {
      expert[lane] = id;
      weight[lane] = w;
    }
    if (!more) return;
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = next[i];
  }
}

// ---------------------------------------------------------------- gradient

// What one slot gives its expert's logit, from its logit xj (id -1: no slot). combine(x) sums
// x over the token's slots, most(x) is the largest of them. base and sum: softmax's
// (weights as they are only).
template <class Sum, class Most>
__device__ __forceinline__ float slot_gradient(const RouteGradArgs& p, int id, float xj, float dw, float base, float sum,
                                               Sum combine, Most most) {
  float v = 0.f;
  if (p.renormalise) {
    const float ls = p.sigmoid ? log_sigmoid(xj) : xj;
    const float top = most(id >= 0 ? ls : -__builtin_inff());
    const float s = id >= 0 && top > -__builtin_inff() ? expf(ls - top) : 0.f;
    const float z = combine(s);
    const float share = s > 0.f ? s / z : 0.f;
    const float mean = combine(id >= 0 ? dw * share : 0.f);
    v = id >= 0 ? share * (dw - mean) : 0.f;
    if (p.sigmoid && id >= 0) v *= 1.f / (1.f + expf(xj));
  } else if (p.sigmoid) {
    // s (1 - s), both factors to their relative accuracy
    if (id >= 0) v = dw * expf(log_sigmoid(xj)) * (1.f / (1.f + expf(xj)));
  } else {
    v = id >= 0 ? dw * (expf(xj - base) / sum) : 0.f;
  }
  return v;
}

// Sigmoids and renormalised weights: only chosen experts have a gradient, the rest of
// the row is zeros. A wave takes 64 / KP tokens (KP >= top_k, a power of two), a lane
// per slot: their rows are cleared first, the slots' gradients formed meanwhile, and
// stored over the zeros when those have arrived. Slots that name one expert
// all hold the sum of theirs, in the slots' order. (16384 tokens of 256 experts, 8
// slots: a wave per token that wrote whole rows 12.5 us, limited by its instructions; this 7.)
template <int KP, bool BF16>
__global__ void __launch_bounds__(kThreads) route_grad_chosen_kernel(RouteGradArgs p) {
  constexpr int TOKENS = 64 / KP, ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane % KP;
  const int bytes = p.E * ES;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 64) * TOKENS;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + wave) * TOKENS; t0 < p.T; t0 += step) {
    const int64_t t = t0 + lane / KP;
    const bool slot = t < p.T && j < p.top_k;
    int id = -1;
    float dw = 0.f, xj = -__builtin_inff();
    if (slot) {
      id = p.expert[t * p.top_k + j];
      dw = p.dweight[t * p.top_k + j];
    }
    for (int r = 0; r < TOKENS && t0 + r < p.T; ++r) {
      char* row = static_cast<char*>(p.dlogits) + (t0 + r) * p.ldd * ES;
      int c = 16 * lane;
      for (; c + 16 <= bytes; c += 1024) *reinterpret_cast<u32x4_any*>(row + c) = u32x4_any{0u, 0u, 0u, 0u};
      for (; c < bytes && c < (bytes & ~15) + 16; c += ES) {  // the lane that the row ends in
        if constexpr (BF16) *reinterpret_cast<uint16_t*>(row + c) = 0;
        else *reinterpret_cast<float*>(row + c) = 0.f;
      }
    }
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) xj = load_logit<BF16>(p.logits, t * p.ldl + id);
    dw = id >= 0 ? p.scale * dw : 0.f;
    const float v = slot_gradient(
        p, id, xj, dw, 0.f, 1.f,
        [](float x) {
#pragma unroll
          for (int o = 1; o < KP; o <<= 1) x += __shfl_xor(x, o);
          return x;
        },
        [](float x) {
#pragma unroll
          for (int o = 1; o < KP; o <<= 1) x = larger(x, __shfl_xor(x, o));
          return x;
        });
    float total = 0.f;
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      const int other = __shfl(id, (lane & ~(KP - 1)) + q);
      const float add = __shfl(v, (lane & ~(KP - 1)) + q);
      total += other == id ? add : 0.f;
    }
    // The zeros have to be there before the values.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (id >= 0) {
      if constexpr (BF16) static_cast<uint16_t*>(p.dlogits)[t * p.ldd + id] = f32_to_bf16_bits(total);
      else static_cast<float*>(p.dlogits)[t * p.ldd + id] = total;
    }
  }
}

// Softmax's weights as they are: every logit has a gradient. A wave per token; lane j
// has slot j while the slots' gradients are formed, then lanes have neighbouring
// experts as in the choice.
template <int EPL, bool BF16>
__global__ void __launch_bounds__(kThreads) route_grad_all_kernel(RouteGradArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float ninf = -__builtin_inff();
  for (int t = blockIdx.x * (kThreads / 64) + wave; t < p.T; t += gridDim.x * (kThreads / 64)) {
    const int64_t row = t * p.ldl;
    int id = -1;
    float dw = 0.f, xj = ninf;
    if (lane < p.top_k) {
      id = p.expert[static_cast<int64_t>(t) * p.top_k + lane];
      dw = p.dweight[static_cast<int64_t>(t) * p.top_k + lane];
    }
    float x[EPL];
    load_row<EPL, BF16>(p.logits, row, p.E, lane, x);
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) xj = load_logit<BF16>(p.logits, row + id);
    dw = id >= 0 ? p.scale * dw : 0.f;
    const bool none = !__any(id >= 0);

    float top = ninf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = x[i] > top ? x[i] : top;
    top = wave_top(top);
    const float base = top == ninf ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      x[i] = fast_exp(x[i] - base);
      sum += x[i];
    }
    sum = wave_sum(sum);
    const float v = slot_gradient(p, id, xj, dw, base, sum, [](float u) { return wave_sum(u); },
                                  [](float u) { return wave_top(u); });

    float d[EPL];
    const float f = none ? 0.f : -wave_sum(v) / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = none ? 0.f : f * x[i];
    const int e0 = lane * EPL;
    for (int j = 0; j < p.top_k; ++j) {
      const int at = __builtin_amdgcn_readlane(id, j) - e0;
      const float add = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
#pragma unroll
      for (int i = 0; i < EPL; ++i) d[i] += i == at ? add : 0.f;
    }

    const int64_t out = t * p.ldd + e0;
    constexpr int WORDS = BF16 ? EPL / 2 : EPL;
    if (WORDS >= 2 && e0 + EPL <= p.E) {
      uint32_t w[WORDS >= 2 ? WORDS : 2];
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        if constexpr (BF16) w[i] = f32x2_to_bf16x2_bits(d[2 * i], d[2 * i + 1]);
        else w[i] = __float_as_uint(d[i]);
      }
      char* at = static_cast<char*>(p.dlogits) + out * (BF16 ? 2 : 4);
      if constexpr (WORDS == 2) *reinterpret_cast<u32x2_any*>(at) = u32x2_any{w[0], w[1]};
#pragma unroll
      for (int h = 0; h < WORDS / 4; ++h)
        *reinterpret_cast<u32x4_any*>(at + 16 * h) = u32x4_any{w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (e0 + i >= p.E) continue;
        if constexpr (BF16) static_cast<uint16_t*>(p.dlogits)[out + i] = f32_to_bf16_bits(d[i]);
        else static_cast<float*>(p.dlogits)[out + i] = d[i];
      }
    }
  }
}

// Workgroups of gemm_route at most: those that are on the card at once.
constexpr int kRouteGrid = 256 * 6;

// Experts per lane for E of them.
template <class Go>
static void with_experts_per_lane(int E, Go go) {
  if (E <= 64) go(std::integral_constant<int, 1>{});
  else if (E <= 128) go(std::integral_constant<int, 2>{});
  else if (E <= 256) go(std::integral_constant<int, 4>{});
  else if (E <= 512) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 16>{});
}

static dim3 token_grid(int T) {
  const int wgs = (T + kThreads / 64 - 1) / (kThreads / 64);
  return dim3(static_cast<unsigned>(wgs < kMaxGrid ? wgs : kMaxGrid));
}

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(std::min((a.T + kThreads / 64 - 1) / (kThreads / 64), kRouteGrid)));
  const auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a); };
  const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_best == 2);
  with_experts_per_lane(a.E, [&](auto n) {
    constexpr int EPL = decltype(n)::value;
    if (scored) bf16 ? run(route_kernel<EPL, true, true>) : run(route_kernel<EPL, false, true>);
    else bf16 ? run(route_kernel<EPL, true, false>) : run(route_kernel<EPL, false, false>);
  });
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, bool bf16, hipStream_t stream) {
  if (a.sigmoid || a.renormalise) {
    // The fewest lanes that hold the slots. 256 experts, 16384 tokens: 8 slots in 8 lanes
    // 6.6 us, in 16 7.2, in 32 12.7; 4 in 4 7.0, in 8 6.2; 2 in 2 7.2, in 4 6.0. 65536
    // tokens: 21.2, 21.2, 36.3; 16.9, 17.0; 13.7, 14.5. (9 to 16 slots take 32 lanes, 12.3
    // and 36 us, where 16 would take 7.6 and 24.)
    const auto run = [&](auto kernel, int kp) {
      hipLaunchKernelGGL(kernel, token_grid((a.T + 64 / kp - 1) / (64 / kp)), dim3(kThreads), 0, stream, a);
    };
    if (a.top_k <= 2) bf16 ? run(route_grad_chosen_kernel<2, true>, 2) : run(route_grad_chosen_kernel<2, false>, 2);
    else if (a.top_k <= 4) bf16 ? run(route_grad_chosen_kernel<4, true>, 4) : run(route_grad_chosen_kernel<4, false>, 4);
    else if (a.top_k <= 8) bf16 ? run(route_grad_chosen_kernel<8, true>, 8) : run(route_grad_chosen_kernel<8, false>, 8);
    else bf16 ? run(route_grad_chosen_kernel<32, true>, 32) : run(route_grad_chosen_kernel<32, false>, 32);
    return hipGetLastError();
  }
  const auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, token_grid(a.T), dim3(kThreads), 0, stream, a); };
  with_experts_per_lane(a.E, [&](auto n) {
    constexpr int EPL = decltype(n)::value;
    bf16 ? run(route_grad_all_kernel<EPL, true>) : run(route_grad_all_kernel<EPL, false>);
  });
  return hipGetLastError();
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
// All of it is latency: 32768 slots of 64 experts take 10.9 us, 131072 of 256 15.9 (a
// first form of waves of their own and a third launch for the scan: 31 and 96). Chunks
// of at least 512, 1024, 2048 or 4096 slots: 9.0, 9.1, 10.9, 17.2 us and 17.1, 17.2, 15.9, 21.3.

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

hipError_t launch_order(const OrderArgs& a, hipStream_t stream) {
  const size_t lds = static_cast<size_t>(a.G + 1) * sizeof(int);
  if (order_small(a.S, a.G)) {
    hipLaunchKernelGGL((order_place_kernel<kSmallWaves, true>), dim3(1), dim3(64 * kSmallWaves), kSmallWaves * lds,
                       stream, a);
    return hipGetLastError();
  }
  // Without slots there are no counts (and no workspace): one workgroup writes the offsets.
  if (a.chunks > 0) {
    hipLaunchKernelGGL(order_count_kernel, dim3(a.chunks), dim3(64 * kOrderWaves), lds, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL((order_place_kernel<kOrderWaves, false>), dim3(a.chunks > 0 ? a.chunks : 1),
                     dim3(64 * kOrderWaves), kOrderWaves * lds, stream, a);
  return hipGetLastError();
}

}  // namespace g355
