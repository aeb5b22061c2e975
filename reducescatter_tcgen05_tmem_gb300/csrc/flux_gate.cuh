// What the forms of the routing with expert groups share: arguments, reductions, and
// the choice in doubles.  Formulas: flux_gate.cu.
#pragma once

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

struct GroupGateArgs {
  const float* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  const int32_t* ids_in;
  const float* dweights;
  float* dlogits;
  int T, E, topk, G, kept, top;
  int n, pad;          // experts of a group; words between groups in shared memory
  int lpg, log_lpg;    // lanes that rank one group
  int per;             // octet form: scores of a lane
  uint32_t div_per;    // ceil(2^20 / per)
  int vecs, trips, rivals;  // wide form: vectors of a lane; of a lane in its group; groups that a lane compares
  int np;              // wide form: places of a group, n up to a multiple of four
  uint32_t div_np;     // ceil(2^20 / np)
  uint32_t div_n;      // ceil(2^20 / n): e / n = e div_n >> 20 for e < 1024
  int row;             // values of a token's row in shared memory
  int softmax, renorm, accumulate;
  float scale;
};

// A warp a token: what a call of it needs beyond the common arguments, and its launch.
flux_status_t group_gate_wide(GroupGateArgs a, const DeviceInfo& dev, cudaStream_t s);

namespace {

constexpr int GG_WARPS = 8, GG_THREADS = GG_WARPS * 32;
constexpr int GG_SMS = 152;
constexpr float G_LOG2E = 1.4426950408889634f;

// What a token needs in shared memory: its values, the picked experts, the groups' ranks
// and the ends of their ranges, the kept groups.
__host__ __device__ inline size_t gate_token_bytes(int row, int topk) { return static_cast<size_t>(row + topk + 4 * 32) * 4; }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sigmoid(x) e^-min(peak, 0), what a chosen score brings to renormalised weights whose
// largest logit is peak; sigmoid(x) with a peak of 0.  1 + e^-|x| is at most 2: rcp of 1 +
// e^-x would be 0 for logits below -87, whose shares fp32 still holds.  (rcp: to one unit
// in the last place, where a rounded quotient costs eight times as much)
__device__ __forceinline__ float sigmoid_share(float x, float peak) {
  return expf(fminf(x, 0.0f) - fminf(peak, 0.0f)) * rcp(1.0f + expf(-fabsf(x)));
}

// Unsigned numbers in the order of the floats (no NaN; 0 is below all of them).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 becomes 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Reductions over the LPT lanes of a token (all lanes of the warp take part).
template <int LPT>
struct Over {
  static __device__ __forceinline__ uint32_t max(uint32_t v) {
    if constexpr (LPT == 32) return __reduce_max_sync(0xFFFFFFFFu, v);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v = ::max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
  static __device__ __forceinline__ uint32_t min(uint32_t v) {
    if constexpr (LPT == 32) return __reduce_min_sync(0xFFFFFFFFu, v);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v = ::min(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
  static __device__ __forceinline__ uint32_t any(uint32_t v) {
    if constexpr (LPT == 32) return __reduce_or_sync(0xFFFFFFFFu, v);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v |= __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
  static __device__ __forceinline__ float maxf(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
};

// Where a group's rank in doubles may lie, from its fp32 rank and the largest values
// that make it (m2 0 where there is one): both values' errors, and their own and the
// sum's rounding.  By the group's own values: a group that is masked with the type's
// lowest value must not widen the others' ranges (131072 tokens with two such groups
// of eight took 2.1 ms that way, every one of them by its choice in doubles; 87 us).  A sum
// that passes fp32 lies past 3.4e38; an infinite value is one in doubles too.
struct RankRange {
  float error, low, high;
  __device__ __forceinline__ RankRange(float rank, float m1, float m2, float unsure) {
    error = fmaf(0x1p-22f, isinf(m1) ? 0.0f : fabsf(m1), fmaf(0x1p-22f, isinf(m2) ? 0.0f : fabsf(m2), unsure));
    const bool past = isinf(rank) && !isinf(m1) && !isinf(m2);
    low = past && rank > 0.0f ? 3.4e38f : rank - error;
    high = past && rank < 0.0f ? -3.4e38f : rank + error;
  }
};
// Whether the kept groups, of which `low` is the least end of a range, and those left out,
// of which `high` is the greatest, are told apart: equal infinite ones are by index.
__device__ __forceinline__ bool ranks_apart(float low, float high) { return low > high || (low == high && isinf(low)); }

// f(e, logit) for the lane's experts of a row, a NaN as -inf.
template <int LPT, typename F>
__device__ __forceinline__ void each_logit(const float* row, int E, int l, F&& f) {
  if (E % 4 == 0) {
#pragma unroll 2
    for (int e = l * 4; e < E; e += LPT * 4) {
      const float4 q = load_global(reinterpret_cast<const float4*>(row + e));
      f(e, fmaxf(q.x, -INFINITY));
      f(e + 1, fmaxf(q.y, -INFINITY));
      f(e + 2, fmaxf(q.z, -INFINITY));
      f(e + 3, fmaxf(q.w, -INFINITY));
    }
  } else {
#pragma unroll 4
    for (int e = l; e < E; e += LPT) f(e, fmaxf(load_global(row + e), -INFINITY));
  }
}

// A token's places in shared memory.
struct Rows {
  float* val;
  int32_t* pick;
  float *rank, *low, *high;
  int32_t* kept;
  __device__ __forceinline__ Rows(char* base, int row, int topk) {
    val = reinterpret_cast<float*>(base);
    pick = reinterpret_cast<int32_t*>(val + row);
    rank = reinterpret_cast<float*>(pick + topk);
    low = rank + 32;
    high = low + 32;
    kept = reinterpret_cast<int32_t*>(high + 32);
  }
};

// Whether a group's rank is made of its two largest values.  Of a group of one there is
// one; without a bias it goes through the same sum, as its score and not as its logit
// (m2 is -inf, whose score is 0): logits may differ where scores are equal.
__device__ __forceinline__ bool ranked_by_two(const GroupGateArgs& a, bool biased) { return a.top == 2 && (a.n > 1 || !biased); }
__device__ __forceinline__ int group_of(const GroupGateArgs& a, int e) { return static_cast<int>((e * a.div_n) >> 20); }
__device__ __forceinline__ int place(const GroupGateArgs& a, int e) { return a.pad == 0 ? e : e + group_of(a, e) * a.pad; }
// The expert at place p of the kept groups' experts in order.
__device__ __forceinline__ int expert_at(const GroupGateArgs& a, const int32_t* kept, int p) {
  if (a.kept == a.G) return p;
  const int q = group_of(a, p);
  return kept[q] * a.n + (p - q * a.n);
}

// Doubles as numbers in their order, for maxima over lanes in halves of 32 bits.
__device__ __forceinline__ unsigned long long order_of(double v) {
  const unsigned long long u = __double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double value_of(unsigned long long k) { return __longlong_as_double(k >> 63 ? k & ~(1ull << 63) : ~k); }
__device__ __forceinline__ unsigned long long largest_of(uint32_t mask, unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(mask, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(mask, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}

// A softmax's sum in doubles, over the LANES lanes of a token; top, its largest logit, is
// finite.  (All lanes of the warp take part.)
template <int LANES>
__device__ __noinline__ double softmax_total64(const float* row, int E, int l, float top) {
  double total = 0.0;
#pragma unroll 4
  for (int e = l; e < E; e += LANES) {
    const float x = load_global(row + e);
    total += exp(static_cast<double>(x != x ? -INFINITY : x) - static_cast<double>(top));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  return total;
}

// An expert's bias, a NaN as -inf: no value of the choice is a NaN, which would stand at
// the head of a list and hide what is behind it.
__device__ __forceinline__ float bias_of(const float* bias, int e) { return fmaxf(load_global(bias + e), -INFINITY); }

// Two values in doubles, side by side: a dependent double operation takes some 100
// cycles on this GPU.  (top and total: of a softmax)
template <bool SOFT>
__device__ __noinline__ double2 biased_scores64(float x, float x_bias, float y, float y_bias, float top, double total) {
  const double p = static_cast<double>(x != x ? -INFINITY : x), q = static_cast<double>(y != y ? -INFINITY : y);
  const double a = exp(SOFT ? p - static_cast<double>(top) : -p), b = exp(SOFT ? q - static_cast<double>(top) : -q);
  const double s = SOFT ? a / total : 1.0 / (1.0 + a), t = SOFT ? b / total : 1.0 / (1.0 + b);
  return make_double2(s + static_cast<double>(x_bias), t + static_cast<double>(y_bias));
}

// The order of a token's chosen experts, one to each of LANES lanes (those from topk on
// have none), and of the one expert left out next to them (-1: none), by their doubles:
// the place of the lane's own in x, of the one left out in y.  Takes 3 us, the choice in
// full 12 to 20.
template <int LANES, bool SOFT>
__device__ __noinline__ int2 order64(const float* row, const float* bias, int e, int out, int l, int topk, float top, double total) {
  const bool here = l < topk;
  const int mine = here ? e : 0, f = out >= 0 ? out : 0;
  const double2 d = biased_scores64<SOFT>(load_global(row + mine), bias_of(bias, mine), load_global(row + f), bias_of(bias, f), top, total);
  auto first = [](double u, int i, double v, int k) { return u > v || (u == v && i < k); };
  int2 place = make_int2(out >= 0 && first(d.y, out, d.x, e), 0);
  for (int j = 0; j < topk; ++j) {
    const double v = __shfl_sync(0xFFFFFFFFu, d.x, j, LANES);
    const int k = __shfl_sync(0xFFFFFFFFu, e, j, LANES);
    place.x += j != l && first(v, k, d.x, e);
    place.y += first(v, k, d.y, out);
  }
  return place;
}

// The choice in doubles, by the LPT lanes of one token (mask).  Writes the kept groups
// and, as pick, the places of the chosen ones among the kept groups'
// experts.  A few tokens in a long batch come here, and the last one holds up the launch:
// a token of 256 experts took 60 us with double comparisons and shuffles of doubles.
template <int LPT>
__device__ __noinline__ void choose64(const GroupGateArgs& a, const float* row, int32_t* kept, int32_t* pick, int l,
                                      uint32_t some) {
  constexpr int MINE = LPT == 32 ? FLUX_MAX_EXPERTS / 32 : 64 / LPT;
  constexpr unsigned long long LEAST = 0x000FFFFFFFFFFFFFull;  // order_of(-inf)
  const uint32_t mask = LPT == 32 ? 0xFFFFFFFFu : some;
  auto logit = [&](int e) {
    const float x = load_global(row + e);
    return static_cast<double>(x != x ? -INFINITY : x);
  };
  double top = -INFINITY, total = 0.0;
  if (a.softmax) {
    for (int e = l; e < a.E; e += LPT) top = fmax(top, logit(e));
    top = value_of(largest_of(mask, order_of(top)));
    for (int e = l; e < a.E; e += LPT) total += isinf(top) ? (logit(e) == top ? 1.0 : 0.0) : exp(logit(e) - top);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) total += __shfl_xor_sync(mask, total, o);
  }
  auto score = [&](double x) {
    if (!a.softmax) return 1.0 / (1.0 + exp(-x));
    return (isinf(top) ? (x == top ? 1.0 : 0.0) : exp(x - top)) / total;
  };
  unsigned long long c[MINE];  // experts l, l + LPT, ...
#pragma unroll 4
  for (int e = l, i = 0; e < a.E; e += LPT, ++i) {
    const double x = logit(e);
    c[i] = order_of(a.bias != nullptr ? score(x) + static_cast<double>(bias_of(a.bias, e)) : x);
  }
  uint32_t in = 0xFFFFFFFFu;
  if (a.kept < a.G) {
    unsigned long long mine[32 / LPT];  // ranks of groups l, l + LPT, ...
#pragma unroll 1
    for (int g = 0; g < a.G; ++g) {
      // the group's two largest: a lane's own first, then over the lanes
      unsigned long long m1 = 0, m2 = 0;
      const int from = g * a.n, to = from + a.n;
#pragma unroll 1
      for (int i = from / LPT; i * LPT < to; ++i) {
        const int e = i * LPT + l;
        if (e < from || e >= to) continue;
        m2 = max(m2, min(m1, c[i]));
        m1 = max(m1, c[i]);
      }
      const unsigned long long best = largest_of(mask, m1);
      double r = value_of(best);
      if (a.top == 2 && a.n > 1) {
        const uint32_t all = __ballot_sync(mask, m1 == best);
        const int owner = (__ffs(all) - 1) % LPT;
        const double second = value_of(largest_of(mask, l == owner ? m2 : m1));
        r = a.bias != nullptr ? r + second : score(r) + score(second);
      } else if (ranked_by_two(a, a.bias != nullptr)) {
        r = score(r);
      }
      if (g % LPT == l) mine[g / LPT] = r != r ? LEAST : order_of(r);
    }
    // the kept ones one after the other, the first of equal ones first
    uint32_t left = 0;
    for (int g = l, i = 0; g < a.G; g += LPT, ++i) left |= 1u << i;
    in = 0;
#pragma unroll 1
    for (int k = 0; k < a.kept; ++k) {
      unsigned long long m = 0;
      for (int i = 0; i < 32 / LPT; ++i)
        if (left >> i & 1u) m = max(m, mine[i]);
      const unsigned long long best = largest_of(mask, m);
      uint32_t g = 0xFFFFFFFFu;
      for (int i = 32 / LPT - 1; i >= 0; --i)
        if ((left >> i & 1u) && mine[i] == best) g = i * LPT + l;
      g = __reduce_min_sync(mask, g);
      if (g % LPT == static_cast<uint32_t>(l)) left &= ~(1u << g / LPT);
      in |= 1u << g;
    }
    for (int g = l; g < a.G; g += LPT)
      if (in >> g & 1u) kept[__popc(in & ((1u << g) - 1u))] = g;
#pragma unroll 1
    for (int e = l, i = 0; e < a.E; e += LPT, ++i)
      if (!(in >> group_of(a, e) & 1u)) c[i] = 0;
    __syncwarp(mask);
  }
  // a lane's best, looked for again when it has been taken
  unsigned long long m;
  int at;
  auto look = [&] {
    m = 0;
    at = 0;
#pragma unroll 1
    for (int e = l, i = 0; e < a.E; e += LPT, ++i)
      if (c[i] > m) {
        m = c[i];
        at = i;
      }
  };
  look();
#pragma unroll 1
  for (int j = 0; j < a.topk; ++j) {
    const unsigned long long best = largest_of(mask, m);
    const int e = __reduce_min_sync(mask, m == best ? static_cast<uint32_t>(at * LPT + l) : 0xFFFFFFFFu);
    if (e % LPT == l) {
      c[at] = 0;
      look();
    }
    if (l == 0) {
      const int g = group_of(a, e);
      pick[j] = a.kept < a.G ? __popc(in & ((1u << g) - 1u)) * a.n + e - g * a.n : e;
    }
    __syncwarp(mask);
  }
}

// The largest of the lanes' numbers; a NaN counts only where there is nothing else.
__device__ __forceinline__ float warp_largest(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace
}  // namespace flux
