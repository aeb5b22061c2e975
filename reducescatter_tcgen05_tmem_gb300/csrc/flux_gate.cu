// Routing to experts with groups: scores, the choice of groups and experts, the
// weights, and the gradient of the scores from the weights' gradient.
//
//   s_e = sigmoid(x_e) or softmax(x)_e
//   c_e = s_e + bias_e                     (the choice alone; x_e itself without a bias)
//   groups of E / G neighbours, ranked by the sum of their 1 or 2 largest c; the best are kept
//   the topk largest c of the kept groups' experts, ties to the lowest index
//   w_j = scale s_j, or scale s_j / sum_i s_i over the chosen
//
// Backward, g_j = scale dw_j, sums over the chosen:
//
//   sigmoid                dx_j = s_j (1 - s_j) g_j
//   sigmoid, renormalised  dx_j = v_j (1 - s_j) (g_j - sum_i v_i g_i),  v = s / sum s
//   softmax, renormalised  dx_j = v_j (g_j - sum_i v_i g_i)
//   softmax                dx_e = p_e ([e chosen] g_e - sum_i p_i g_i)   for every expert
//
// The choice is that of the double precision values: fp32 cannot tell neighbours in
// rank apart often enough (one token in a thousand at 256 experts).  The kernel
// chooses in fp32, whose error it bounds; where two neighbours in the order, or the
// last one in and the first one out, are closer than the bounds it makes that
// token's choice again in doubles.  Values made from equal scores and equal biases
// are equal in both, so that ties cost nothing extra.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int GG_WARPS = 8, GG_THREADS = GG_WARPS * 32;
constexpr int GG_SMS = 152;
constexpr float G_LOG2E = 1.4426950408889634f;

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

// What a token needs in shared memory: its values, the picked experts, the groups'
// ranks, the ranks in order, the kept groups.
__host__ __device__ inline size_t gate_token_bytes(int row, int topk) { return static_cast<size_t>(row + topk + 3 * 32) * 4; }

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

// Whether the last kept group and the first one left out are told apart by their fp32
// ranks: by more than their errors, or equal and infinite where nothing finite is so
// large that its sum may have become so (then `room` is infinite too).
__device__ __forceinline__ bool ranks_apart(float last, float next, float room) {
  return last - next > room || (last == next && isinf(last) && room < INFINITY);
}

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
  float *rank, *sorted;
  int32_t* kept;
  __device__ __forceinline__ Rows(char* base, int row, int topk) {
    val = reinterpret_cast<float*>(base);
    pick = reinterpret_cast<int32_t*>(val + row);
    rank = reinterpret_cast<float*>(pick + topk);
    sorted = rank + 32;
    kept = reinterpret_cast<int32_t*>(sorted + 32);
  }
};

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
  const double2 d = biased_scores64<SOFT>(load_global(row + mine), load_global(bias + mine), load_global(row + f), load_global(bias + f), top, total);
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
// experts.  One token in a thousand comes here, and the last one holds up the launch:
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
    const double x = logit(e), v = a.bias != nullptr ? score(x) + static_cast<double>(load_global(a.bias + e)) : x;
    c[i] = v != v ? LEAST : order_of(v);
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

// One token of up to 64 experts to eight lanes, NC candidates each.  The lanes put the
// values into a row of shared memory, rank the groups from there, and take their
// candidates (those of the kept groups, in order) into registers for topk rounds of a
// maximum.  For long batches of what the octet form does not take: 131072 tokens, 4 of 48
// experts in 6 of 16 groups 82 us, a warp a token 108; 10 of 16 experts 31 and 55.
template <int NC>
__global__ void __launch_bounds__(GG_THREADS, 5)
group_gate_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int LPT = 8, TPW = 32 / LPT;
  extern __shared__ uint4 smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPT, sub = lane / LPT;
  using O = Over<LPT>;
  const Rows r(reinterpret_cast<char*>(smem) + (warp * TPW + sub) * gate_token_bytes(a.row, a.topk), a.row, a.topk);
  const bool grouped = a.kept < a.G, biased = a.bias != nullptr;
  const bool soft_row = a.softmax && (biased || !a.renorm || (grouped && a.top == 2));
  wait_for_previous();
  for (long long t0 = static_cast<long long>(blockIdx.x * GG_WARPS + warp) * TPW; t0 < a.T; t0 += static_cast<long long>(gridDim.x) * GG_WARPS * TPW) {
    const bool here = t0 + sub < a.T;
    const size_t t = static_cast<size_t>(here ? t0 + sub : a.T - 1);
    const float* row = a.logits + t * a.E;
    __syncwarp();
    float top = -INFINITY, inv = 1.0f, total = 1.0f;
    auto soft = [&](float x) { return isinf(top) ? (x == top ? 1.0f : 0.0f) : ex2((x - top) * G_LOG2E); };
    auto score = [&](float x) { return a.softmax ? soft(x) * inv : rcp(1.0f + ex2(-x * G_LOG2E)); };
    // the values: x without a bias, else s + bias
    if (soft_row) {
      each_logit<LPT>(row, a.E, l, [&](int e, float x) {
        r.val[place(a, e)] = x;
        top = fmaxf(top, x);
      });
      top = O::maxf(top);
      total = 0.0f;
      auto second = [&](int e) {
        const int at = place(a, e);
        const float v = soft(r.val[at]);
        total += v;
        if (biased) r.val[at] = v;
      };
      if (a.E % 4 == 0) {
        for (int e = l * 4; e < a.E; e += LPT * 4) second(e), second(e + 1), second(e + 2), second(e + 3);
      } else {
        for (int e = l; e < a.E; e += LPT) second(e);
      }
      total = O::sum(total);
      inv = rcp(total);
      if (biased) {
        auto third = [&](int e) {
          const int at = place(a, e);
          r.val[at] = fmaxf(r.val[at] * inv + load_global(a.bias + e), -INFINITY);
        };
        if (a.E % 4 == 0) {
          for (int e = l * 4; e < a.E; e += LPT * 4) third(e), third(e + 1), third(e + 2), third(e + 3);
        } else {
          for (int e = l; e < a.E; e += LPT) third(e);
        }
      }
    } else {
      each_logit<LPT>(row, a.E, l, [&](int e, float x) {
        r.val[place(a, e)] = biased ? fmaxf(score(x) + load_global(a.bias + e), -INFINITY) : x;
      });
    }
    __syncwarp();
    // How far apart two values have to be for their order to be sure: errors of the
    // sigmoid 4.4 2^-24 (argument, ex2, sum, reciprocal), of the softmax 70 2^-24 of its
    // largest, and half an ulp for the bias; twice that for two values, and a margin.  Of
    // softmax ranks without a bias 5 2^-24 for each of four values: the error of their
    // sum, most of the 70, is a factor that they share.
    const float unsure = a.softmax ? (biased ? 0x1p-16f : 0x1p-20f) * inv : 0x1p-20f;
    uint32_t doubt = 0;  // the groups' choice is not sure
    if (grouped) {
      const int per = LPT / a.lpg;
      float big = 0.0f;
      for (int g0 = 0; g0 < a.G; g0 += per) {
        const int g = g0 + l / a.lpg;
        float m1 = -INFINITY, m2 = -INFINITY;
        if (g < a.G) {
          const float* v = r.val + g * (a.n + a.pad);
          for (int i = l % a.lpg; i < a.n; i += a.lpg) {
            m2 = fmaxf(m2, fminf(m1, v[i]));
            m1 = fmaxf(m1, v[i]);
          }
        }
        for (int o = a.lpg / 2; o > 0; o >>= 1) {
          const float o1 = __shfl_xor_sync(0xFFFFFFFFu, m1, o), o2 = __shfl_xor_sync(0xFFFFFFFFu, m2, o);
          m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
          m1 = fmaxf(m1, o1);
        }
        if (a.top == 2 && a.n > 1) {
          if (!biased) m1 = score(m1), m2 = score(m2);
          if (g < a.G) big = fmaxf(big, (isinf(m1) ? 0.0f : fabsf(m1)) + (isinf(m2) ? 0.0f : fabsf(m2)));
          m1 = fmaxf(m1 + m2, -INFINITY);
        } else if (g < a.G && !isinf(m1)) {
          big = fmaxf(big, fabsf(m1));
        }
        if (g < a.G && l % a.lpg == 0) r.rank[g] = m1;
      }
      __syncwarp();
      uint32_t in = 0;
      for (int g = l; g < a.G; g += LPT) {
        const float mine = r.rank[g];
        int pos = 0;
        for (int o = 0; o < a.G; ++o) {
          const float other = r.rank[o];
          pos += other > mine || (other == mine && o < g);
        }
        r.sorted[pos] = mine;
        if (pos < a.kept) in |= 1u << g;
      }
      in = O::any(in);
      for (int g = l; g < a.G; g += LPT)
        if (in >> g & 1u) r.kept[__popc(in & ((1u << g) - 1u))] = g;
      big = O::maxf(big);
      __syncwarp();
      // (ranks that are logits are exact)
      if (biased || (a.top == 2 && a.n > 1))
        doubt = !ranks_apart(r.sorted[a.kept - 1], r.sorted[a.kept], 2.0f * unsure + 0x1p-21f * big);
    }
    const int count = a.kept * a.n;
    uint32_t key[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * LPT + l;
      key[i] = p < count ? order_of(r.val[place(a, expert_at(a, r.kept, p))]) : 0u;
    }
    for (int j = 0; j < a.topk; ++j) {
      uint32_t m = key[0];
#pragma unroll
      for (int i = 1; i < NC; ++i) m = max(m, key[i]);
      const uint32_t best = O::max(m);
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = NC - 1; i >= 0; --i)
        if (key[i] == best) at = i * LPT + l;
      at = O::min(at);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (at == static_cast<uint32_t>(i * LPT + l)) key[i] = 0u;
      if (l == 0) r.pick[j] = static_cast<int>(at);
    }
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NC; ++i) m = max(m, key[i]);
    m = O::max(m);  // the best one left, 0 if none is
    __syncwarp();
    auto expert = [&](int j) { return expert_at(a, r.kept, r.pick[j]); };
    if (biased) {
      auto apart = [&](float hi, float lo) { return hi - lo > unsure + 0x1p-23f * (fabsf(hi) + fabsf(lo)); };
      auto same = [&](int e, int f) { return load_global(row + e) == load_global(row + f) && load_global(a.bias + e) == load_global(a.bias + f); };
      const float last = r.val[place(a, expert(a.topk - 1))];
      uint32_t close = m != 0u && !apart(last, value_of(m));
      for (int j = l; j + 1 < a.topk; j += LPT) close |= !apart(r.val[place(a, expert(j))], r.val[place(a, expert(j + 1))]);
      if (O::any(close)) {
        // equal inputs have equal values: their order is that of the indexes
        uint32_t wrong = 0;
        for (int j = l; j + 1 < a.topk; j += LPT) {
          const int e = expert(j), f = expert(j + 1);
          wrong |= !apart(r.val[place(a, e)], r.val[place(a, f)]) && !same(e, f);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (key[i] != 0u && !apart(last, value_of(key[i])))
            wrong |= !same(expert(a.topk - 1), expert_at(a, r.kept, i * LPT + l));
        doubt |= wrong;
      }
    }
    doubt = O::any(doubt);
    if (doubt) choose64<LPT>(a, row, r.kept, r.pick, l, LPT == 32 ? 0xFFFFFFFFu : ((1u << LPT % 32) - 1u) << (sub * LPT));
    __syncwarp();
    // the weights
    auto chosen = [&](int j) { return fmaxf(load_global(row + expert(j)), -INFINITY); };
    float peak = -INFINITY;
    if (a.renorm) {
      for (int j = l; j < a.topk; j += LPT) peak = fmaxf(peak, chosen(j));
      peak = O::maxf(peak);
    }
    // renormalised sigmoids are scaled by e^-min(peak, 0): very low scores still have shares
    auto weight = [&](float x) {
      if (a.renorm && (a.softmax ? isinf(peak) : peak == -INFINITY)) return x == peak ? 1.0f : 0.0f;
      if (a.softmax) return a.renorm ? expf(x - peak) : isinf(top) ? soft(x) : expf(x - top);
      return expf(fminf(x, 0.0f) - (a.renorm ? fminf(peak, 0.0f) : 0.0f)) / (1.0f + expf(-fabsf(x)));
    };
    float sum = a.softmax ? total : 1.0f;
    if (a.renorm) {
      sum = 0.0f;
      for (int j = l; j < a.topk; j += LPT) sum += weight(chosen(j));
      sum = O::sum(sum);
    }
    if (here) {
      for (int j = l; j < a.topk; j += LPT) {
        a.ids[t * a.topk + j] = expert(j);
        a.weights[t * a.topk + j] = a.scale * (weight(chosen(j)) / sum);
      }
    }
  }
}

// The largest of the lanes' numbers; a NaN counts only where there is nothing else.
__device__ __forceinline__ float warp_largest(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A token's words in shared memory, wide form: its logits as they come and those of
// the next token (rows of whole vectors for every lane), its values (with groups),
// the picked places, the kept groups, the lists and the order of what they hold.
__host__ __device__ inline int wide_words(int vecs, int row, int topk, int lists) {
  return 2 * 128 * vecs + row + ((topk + 3) & ~3) + 32 + lists * 32 * 6;
}

// One token to a warp, vectors of four experts to a lane, the next token's logits on
// their way while this one's are at work.  The candidates (all experts, or the kept
// groups') lie in LISTS sorted lists of four a lane, so that a round of the choice
// is a maximum over the lists' heads and over the warp, and a shift of the winner's
// list.  Groups begin at multiples of four places; the places behind an odd group's last
// expert hold -inf and are no candidates.
//
// Bound by the length of that chain: 13 tokens of 256 experts 2.9 us in a captured
// graph, 4096 tokens 10 us with cold caches where a token of them needs doubles, 6 where
// none does; 131072 tokens 116 us, which is why long batches take the octet form.
template <int VECS, int LISTS, bool GROUPED, bool SOFT, bool BIASED>
__global__ void __launch_bounds__(GG_THREADS, LISTS <= 2 ? 4 : 3)
group_gate_wide_kernel(const __grid_constant__ GroupGateArgs a) {
  extern __shared__ uint4 smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), vecs = VECS > 0 ? VECS : a.vecs, wide = 128 * vecs;
  float* bias = reinterpret_cast<float*>(smem);
  float* raw2 = bias + (BIASED ? wide : 0) + warp * wide_words(vecs, a.row, a.topk, LISTS);
  float* val = raw2 + 2 * wide;
  int32_t* pick = reinterpret_cast<int32_t*>(val + a.row);
  int32_t* kept = pick + ((a.topk + 3) & ~3);
  float* list = reinterpret_cast<float*>(kept + 32);
  uint32_t* order = reinterpret_cast<uint32_t*>(list + LISTS * 32 * 5);
  const bool two = a.top == 2 && a.n > 1;
  const bool soft_row = SOFT && (BIASED || !a.renorm || (GROUPED && two));
  // experts and their places; a place that holds none is -inf everywhere
  const int shift = a.np - a.n, places = a.G * a.np;
  auto group_of = [&](int p) { return static_cast<int>((p * a.div_np) >> 20); };
  auto place_of = [&](int e) { return e + static_cast<int>((e * a.div_n) >> 20) * shift; };
  auto id_of = [&](int p) { return p - group_of(p) * shift; };
  auto spot = [&](int p) { return a.pad == 0 ? p : p + group_of(p) * a.pad; };  // in val
  auto kept_place = [&](int p) {  // of the kept groups' places in order
    if (a.kept == a.G) return p;
    const int q = group_of(p);
    return kept[q] * a.np + (p - q * a.np);
  };
  const bool whole = a.E % 4 == 0 && shift == 0;  // rows are vectors, and groups too
  for (int p = lane; p < wide; p += 32) {
    if (p >= places || p - group_of(p) * a.np >= a.n) raw2[p] = raw2[wide + p] = -INFINITY;
  }
  for (int q = 0; q < LISTS; ++q) list[(q * 32 + lane) * 5 + 4] = NAN;
  wait_for_previous();
  if constexpr (BIASED) {
    for (int p = threadIdx.x; p < wide; p += GG_THREADS)
      bias[p] = p < places && p - group_of(p) * a.np < a.n ? load_global(a.bias + id_of(p)) : -INFINITY;
    __syncthreads();
  }
  auto fetch = [&](long long at, float* dst) {
    if (at < a.T) {
      const float* src = a.logits + static_cast<size_t>(at) * a.E;
      if (whole) {
#pragma unroll
        for (int v = 0; v < vecs; ++v) {
          const int e = v * 128 + lane * 4;
          if (e < a.E) copy16_async(dst + e, src + e);
        }
      } else {
        for (int e = lane; e < a.E; e += 32) copy4_async(dst + place_of(e), src + e);
      }
    }
    copy_commit();
  };
  const long long step = static_cast<long long>(gridDim.x) * GG_WARPS;
  long long t = static_cast<long long>(blockIdx.x) * GG_WARPS + warp;
  fetch(t, raw2);
  for (int turn = 0; t < a.T; t += step, turn ^= 1) {
    float* raw = raw2 + turn * wide;
    __syncwarp();  // the other row's readers are done
    fetch(t + step, raw2 + (turn ^ 1) * wide);
    copy_wait<1>();
    if (!whole) __syncwarp();  // (vectors are read by the lanes that copied them)
    auto four = [&](int e) {
      float4 x = *reinterpret_cast<const float4*>(raw + e);
      x.x = fmaxf(x.x, -INFINITY), x.y = fmaxf(x.y, -INFINITY), x.z = fmaxf(x.z, -INFINITY), x.w = fmaxf(x.w, -INFINITY);
      return x;
    };
    float top = -INFINITY, inv = 1.0f, total = 1.0f;
    auto soft = [&](float x) { return isinf(top) ? (x == top ? 1.0f : 0.0f) : ex2((x - top) * G_LOG2E); };
    auto score = [&](float x) {
      if constexpr (SOFT) return soft(x) * inv;
      else return rcp(1.0f + ex2(-x * G_LOG2E));
    };
    if (soft_row) {
      for (int v = 0; v < vecs; ++v) {
        const float4 x = four(v * 128 + lane * 4);
        top = fmaxf(top, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
      }
      top = warp_largest(top);
      total = 0.0f;
      for (int v = 0; v < vecs; ++v) {
        const float4 x = four(v * 128 + lane * 4);
        total += (soft(x.x) + soft(x.y)) + (soft(x.z) + soft(x.w));
      }
      total = top == -INFINITY ? static_cast<float>(a.E) : warp_sum(total);
      inv = rcp(total);
    }
    // the values: the logits without a bias, else s + bias
    auto values = [&](int e) {
      float4 x = four(e);
      if constexpr (BIASED) {
        const float4 b = *reinterpret_cast<const float4*>(bias + e);
        x.x = score(x.x) + b.x, x.y = score(x.y) + b.y, x.z = score(x.z) + b.z, x.w = score(x.w) + b.w;
      }
      return x;
    };
    // (how far apart: as in group_gate_kernel)
    const float unsure = SOFT ? (BIASED ? 0x1p-16f : 0x1p-20f) * inv : 0x1p-20f;
    bool doubt = false;
    if constexpr (GROUPED) {
#pragma unroll 2
      for (int v = 0; v < vecs; ++v) {
        const int e = v * 128 + lane * 4;
        *reinterpret_cast<float4*>(val + spot(e)) = values(e);
      }
      __syncwarp();
      // lpg lanes a group
      const int g = lane >> a.log_lpg, sub = lane & (a.lpg - 1);
      float m1 = -INFINITY, m2 = -INFINITY;
      const float* mine = val + g * (a.np + a.pad);
#pragma unroll 2
      for (int k = 0; k < a.trips; ++k) {
        const int i = (k * a.lpg + sub) * 4;
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (g < a.G && i < a.np) q = *reinterpret_cast<const float4*>(mine + i);
        const float p = fmaxf(q.x, q.y), s = fminf(q.x, q.y), u = fmaxf(q.z, q.w), w = fminf(q.z, q.w);
        m2 = fmaxf(fmaxf(m2, fminf(m1, fmaxf(p, u))), fmaxf(fminf(p, u), fmaxf(s, w)));
        m1 = fmaxf(m1, fmaxf(p, u));
      }
      for (int o = a.lpg >> 1; o > 0; o >>= 1) {
        const float o1 = __shfl_xor_sync(0xFFFFFFFFu, m1, o), o2 = __shfl_xor_sync(0xFFFFFFFFu, m2, o);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      const float x1 = m1, x2 = m2;  // (logits without a bias)
      if (!two) m2 = 0.0f;
      else if (!BIASED) m1 = score(m1), m2 = score(m2);
      // the groups before this one in the order, counted by its lanes
      const float rank = g < a.G ? fmaxf(m1 + m2, -INFINITY) : -INFINITY;
      int before = 0;
      for (int k = 0; k < a.rivals; ++k) {
        const int o = k * a.lpg + sub;
        const float other = __shfl_sync(0xFFFFFFFFu, rank, o << a.log_lpg);
        before += o < a.G && (other > rank || (other == rank && o < g));
      }
      for (int o = a.lpg >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
      bool in = g < a.G && before < a.kept;
      if (BIASED || two) {
        const float big = g < a.G ? (isinf(m1) ? 0.0f : fabsf(m1)) + (isinf(m2) ? 0.0f : fabsf(m2)) : 0.0f;
        const float last = -warp_largest(in ? -rank : NAN), next = warp_largest(in || g >= a.G ? NAN : rank);
        const float room = 2.0f * unsure + 0x1p-21f * warp_largest(big);
        doubt = !ranks_apart(last, next, room);
        // Groups next to the border: their ranks in doubles, from their two largest values
        // (unless a third is next to the second) or their largest, wherever they lie.
        if (doubt && !(SOFT && isinf(top))) {
          const double sum = SOFT ? softmax_total64<32>(a.logits + static_cast<size_t>(t) * a.E, a.E, lane, top) : 0.0;
          const bool near = g < a.G && (room == INFINITY || (in ? rank - next <= room : last - rank <= room));
          bool told = near;
          double exact;
          if constexpr (BIASED) {
            const float least = (two ? m2 : m1) - room;
            int count = 0, e = 0, f = 0;
            if (near) {
              for (int k = 0; k < a.trips; ++k) {
                const int i = (k * a.lpg + sub) * 4;
                for (int j = i; j < min(i + 4, a.n); ++j) {
                  if (mine[j] < least) continue;
                  ++count;
                  f = e;
                  e = g * a.np + j;
                }
              }
            }
            int all = count;
            for (int o = a.lpg >> 1; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
            told = near && all == (two ? 2 : 1);
            const double2 d = biased_scores64<SOFT>(raw[e], bias[e], raw[f], bias[f], top, sum);
            exact = (count > 0 ? d.x : 0.0) + (count > 1 ? d.y : 0.0);
            for (int o = a.lpg >> 1; o > 0; o >>= 1) exact += __shfl_xor_sync(0xFFFFFFFFu, exact, o);
          } else {
            const double2 d = biased_scores64<SOFT>(x1, 0.0f, x2, 0.0f, top, sum);
            exact = d.x + d.y;
          }
          exact = told ? fmax(exact, static_cast<double>(-INFINITY)) : rank;
          int ahead = 0;
          for (int o = 0; o < a.G; ++o) {
            const double other = __shfl_sync(0xFFFFFFFFu, exact, o << a.log_lpg);
            ahead += other > exact || (other == exact && o < g);
          }
          if (!__any_sync(0xFFFFFFFFu, near && !told)) {
            in = g < a.G && ahead < a.kept;
            doubt = false;
          }
        }
      }
      const uint32_t set = __ballot_sync(0xFFFFFFFFu, in && sub == 0);
      if (in && sub == 0) kept[__popc(set & ((1u << lane) - 1u))] = g;
      __syncwarp();
    }
    // lists of four, largest first, equal ones in order; their numbers in the bytes of a
    // word, and a NaN at their end
    const int count = a.kept * a.np;
    float h[LISTS];  // the heads
    int at[LISTS];   // and their places
#pragma unroll
    for (int q = 0; q < LISTS; ++q) {
      const int p = q * 128 + lane * 4;
      float4 x = make_float4(NAN, NAN, NAN, NAN);
      if constexpr (GROUPED) {
        if (p < count) {
          const int g = group_of(p);
          x = *reinterpret_cast<const float4*>(val + kept[g] * (a.np + a.pad) + (p - g * a.np));
        }
      } else if (q < vecs) {
        const float4 y = values(p);
        if (p < count) x = y;
      }
      float v[4] = {x.x, x.y, x.z, x.w};
      if (shift != 0) {
        const int left = a.n - (p - group_of(p) * a.np);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? v[i] : NAN;
      }
      uint32_t id[4] = {0, 1, 2, 3};
      auto sort2 = [&](int i) {  // neighbours, if out of order: equal ones stay in theirs
        const bool swap = v[i] < v[i + 1];
        const float hi = swap ? v[i + 1] : v[i], lo = swap ? v[i] : v[i + 1];
        const uint32_t first = swap ? id[i + 1] : id[i], second = swap ? id[i] : id[i + 1];
        v[i] = hi, v[i + 1] = lo, id[i] = first, id[i + 1] = second;
      };
      sort2(0), sort2(1), sort2(2), sort2(0), sort2(1), sort2(0);
      at[q] = (q * 32 + lane) * 5;
#pragma unroll
      for (int i = 1; i < 4; ++i) list[at[q] + i] = v[i];
      list[at[q]] = h[q] = v[0];
      order[q * 32 + lane] = id[0] | id[1] << 8 | id[2] << 16 | id[3] << 24;
    }
    auto head = [&] {
      float m = h[0];
#pragma unroll
      for (int q = 1; q < LISTS; ++q) m = fmaxf(m, h[q]);
      return m;
    };
    // the place among the candidates of what a list holds at `where`
    auto candidate = [&](int where) {
      const int of = static_cast<int>(static_cast<uint32_t>(where) * 52429u >> 18);  // / 5
      return of * 4 + (order[of] >> (where - of * 5) * 8 & 3u);
    };
    // One round after the other.  Where the largest is in several lists, the one with the
    // first expert has it.  To see that costs half a round, so all of them take it; more
    // taken than rounds tell, and the rounds are gone through again with care.
    for (int j0 = 0; j0 < a.topk; j0 += 8) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (j0 + u >= a.topk) break;
        const float best = warp_largest(head());
#pragma unroll
        for (int q = 0; q < LISTS; ++q) {
          if (h[q] == best) {
            pick[j0 + u] = at[q];
            h[q] = list[++at[q]];
          }
        }
      }
    }
    int taken = 0;
#pragma unroll
    for (int q = 0; q < LISTS; ++q) taken += at[q] - (q * 32 + lane) * 5;
    if (__reduce_add_sync(0xFFFFFFFFu, taken) != a.topk) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        at[q] = (q * 32 + lane) * 5;
        h[q] = list[at[q]];
      }
      for (int j = 0; j < a.topk; ++j) {
        const float best = warp_largest(head());
        uint32_t first = 0xFFFFFFFFu;
#pragma unroll
        for (int q = LISTS - 1; q >= 0; --q)
          if (h[q] == best) first = candidate(at[q]);
        const uint32_t p = __reduce_min_sync(0xFFFFFFFFu, first);
#pragma unroll
        for (int q = 0; q < LISTS; ++q) {
          if (h[q] == best && p == first && p / 128 == q) {
            pick[j] = at[q];
            h[q] = list[++at[q]];
          }
        }
      }
    }
    __syncwarp();
    const bool few = a.topk <= 32;
    auto expert = [&](int p) { return GROUPED ? kept_place(p) : p; };  // (its place)
    int own = few && lane < a.topk ? candidate(pick[lane]) : 0;
    if (!few) {
      for (int j = lane; j < a.topk; j += 32) pick[j] = candidate(pick[j]);
      __syncwarp();
    }
    own = expert(own);
    if constexpr (BIASED) {
      const float next = warp_largest(head());  // the best one left, NaN if none is
      auto value = [&](int e) { return GROUPED ? val[spot(e)] : score(fmaxf(raw[e], -INFINITY)) + bias[e]; };
      auto apart = [&](float hi, float lo) { return hi - lo > unsure + 0x1p-23f * (fabsf(hi) + fabsf(lo)); };
      bool close = false;
      if (few) {
        const float hi = value(own), after = __shfl_down_sync(0xFFFFFFFFu, hi, 1);
        const float lo = lane + 1 < a.topk ? after : next;
        close = lane < a.topk && lo == lo && !apart(hi, lo);
      } else {
        for (int j = lane; j < a.topk; j += 32) {
          const float lo = j + 1 < a.topk ? value(expert(pick[j + 1])) : next;
          close |= lo == lo && !apart(value(expert(pick[j])), lo);
        }
      }
      if (__any_sync(0xFFFFFFFFu, close)) {
        // equal inputs have equal values: their order is that of the indexes
        auto same = [&](int e, int f) { return raw[e] == raw[f] && bias[e] == bias[f]; };
        auto picked = [&](int j) { return expert(few ? candidate(pick[j]) : pick[j]); };
        const int end = picked(a.topk - 1);
        bool unsorted = false;
        for (int j = lane; j + 1 < a.topk; j += 32) {
          const int e = picked(j), f = picked(j + 1);
          if (!apart(value(e), value(f))) unsorted |= !same(e, f);
        }
        // and what was left out next to the last one in
        uint32_t out = 0xFFFFFFFFu, others = 0, equal = 0;
#pragma unroll
        for (int q = 0; q < LISTS; ++q) {
          for (int i = at[q]; i < (q * 32 + lane) * 5 + 4; ++i) {
            if (list[i] != list[i] || apart(value(end), list[i])) continue;
            const int f = expert(candidate(i));
            if (same(end, f)) {
              ++equal;
            } else {
              ++others;
              out = f;
            }
          }
        }
        others = __reduce_add_sync(0xFFFFFFFFu, others);
        out = __reduce_min_sync(0xFFFFFFFFu, out);
        equal = __reduce_add_sync(0xFFFFFFFFu, equal);
        unsorted = __any_sync(0xFFFFFFFFu, unsorted) || others > 0u;
        if (unsorted && !(SOFT && isinf(top)) && few && others <= 1u && equal == 0u) {
          // two neighbours, or the last one in and the first one out: by their doubles alone
          const int f = others == 1u ? static_cast<int>(out) : -1;
          const float* row = a.logits + static_cast<size_t>(t) * a.E;
          const double sum = SOFT ? softmax_total64<32>(row, a.E, lane, top) : 0.0;
          const int2 place = order64<32, SOFT>(row, a.bias, id_of(own), f < 0 ? f : id_of(f), lane, a.topk, top, sum);
          __syncwarp();
          if (lane < a.topk && place.x < a.topk) pick[place.x] = own;
          if (lane == 0 && f >= 0 && place.y < a.topk) pick[place.y] = f;
          __syncwarp();
          if (lane < a.topk) own = pick[lane];
        } else {
          doubt |= unsorted;
        }
      }
    }
    if ((BIASED || GROUPED) && __any_sync(0xFFFFFFFFu, doubt)) {
      choose64<32>(a, a.logits + static_cast<size_t>(t) * a.E, kept, pick, lane, 0xFFFFFFFFu);
      auto chosen = [&](int j) { return place_of(expert_at(a, kept, pick[j])); };
      if (few) {
        if (lane < a.topk) own = chosen(lane);
      } else {  // as places among the kept groups' again
        for (int j = lane; j < a.topk; j += 32) pick[j] = place_of(pick[j]);
        __syncwarp();
      }
    }
    // The weights, with the rules of group_gate_kernel.  rcp: to one unit in the last
    // place, where a rounded quotient costs eight times as much.
    auto logit = [&](int e) { return fmaxf(raw[e], -INFINITY); };
    float peak = 0.0f;
    auto weight = [&](float x) {
      if constexpr (SOFT) {
        if (a.renorm) return isinf(peak) ? (x == peak ? 1.0f : 0.0f) : expf(x - peak);
        return isinf(top) ? (x == top ? 1.0f : 0.0f) : expf(x - top);
      } else {
        if (!a.renorm || peak > -64.0f) return rcp(1.0f + expf(-x));
        if (peak == -INFINITY) return 1.0f;
        return expf(x - peak);  // so low that 1 + e^x is 1
      }
    };
    int32_t* ids = a.ids + static_cast<size_t>(t) * a.topk;
    float* weights = a.weights + static_cast<size_t>(t) * a.topk;
    if (few) {
      const bool here = lane < a.topk;
      const float x = here ? logit(own) : -INFINITY;
      if (a.renorm) peak = warp_largest(x);
      float w = weight(x);
      w = here ? w : 0.0f;
      const float sum = a.renorm ? warp_sum(w) : total;
      if (here) {
        ids[lane] = id_of(own);
        weights[lane] = a.scale * w * rcp(sum);
      }
    } else {
      float sum = total;
      if (a.renorm) {
        peak = -INFINITY;
        for (int j = lane; j < a.topk; j += 32) peak = fmaxf(peak, logit(expert(pick[j])));
        peak = warp_largest(peak);
        sum = 0.0f;
        for (int j = lane; j < a.topk; j += 32) sum += weight(logit(expert(pick[j])));
        sum = warp_sum(sum);
      }
      for (int j = lane; j < a.topk; j += 32) {
        const int e = expert(pick[j]);
        ids[j] = id_of(e);
        weights[j] = a.scale * weight(logit(e)) * rcp(sum);
      }
    }
  }
  copy_wait<0>();
}

// Words of a lane in shared memory, octet form: its logits, then its sorted lists of
// four (values, a NaN, their order; 8-byte stores).  No two of the eight lanes that read
// 16 bytes at a time meet in a bank.
template <int P>
__host__ __device__ constexpr int octet_pitch() {
  return P == 32 ? 52 : P == 16 ? 28 : 12;
}
__host__ __device__ inline int octet_words(int pitch) { return 32 * pitch + 4 * 8 + 8 + 32; }

// Four tokens to a warp: a token's scores lie in neighbouring order in eight lanes, P
// at most in each, so that a group is one lane (or 2, 4 or 8) and most of the work is
// in the lanes' own registers.  Lists and rounds as in group_gate_wide_kernel.
// 131072 x 256 (8 of 256 in 4 of 8 groups) 80 us, of which the logits' bytes need 20:
// bound by issue slots (62 % busy with the 24 warps an SM that 80 registers leave) and
// by tokens that need doubles.
template <int P, bool SOFT, bool BIASED>
__global__ void __launch_bounds__(GG_THREADS, P == 32 ? 3 : 4)
group_gate_octet_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int LISTS = P / 4, S = octet_pitch<P>();
  extern __shared__ uint4 smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), l = lane & 7, sub = lane >> 3;
  float* bias = reinterpret_cast<float*>(smem);  // [8][P + 4], as the lanes hold the scores
  float* mem = bias + (BIASED ? 8 * (P + 4) : 0) + warp * octet_words(S);
  float* own = mem + lane * S;
  int32_t* pick = reinterpret_cast<int32_t*>(mem + 32 * S) + sub * 8;
  int32_t* pick64 = reinterpret_cast<int32_t*>(mem + 32 * S) + 4 * 8;
  int32_t* kept64 = pick64 + 8;
  using O = Over<8>;
  const bool grouped = a.kept < a.G, two = a.top == 2 && a.n > 1;
  const bool soft_row = SOFT && (BIASED || !a.renorm || (grouped && two));
  const int mine = min(a.per, max(a.E - l * a.per, 0));  // scores of this lane
  const bool full = a.per == P && a.E == 8 * P;
  const int group = l >> a.log_lpg, lpg = 1 << a.log_lpg;
  wait_for_previous();
  if constexpr (BIASED) {
    for (int i = threadIdx.x; i < 8 * (P + 4); i += GG_THREADS) {
      const int b = i / (P + 4), k = i - b * (P + 4), e = b * a.per + k;
      bias[i] = k < a.per && e < a.E ? load_global(a.bias + e) : -INFINITY;
    }
    __syncthreads();
  }
  const long long step = static_cast<long long>(gridDim.x) * GG_WARPS * 4;
  for (long long first = static_cast<long long>(blockIdx.x) * GG_WARPS * 4; first < a.T; first += step) {
    const bool token = first + warp * 4 + sub < a.T;
    const long long t = token ? first + warp * 4 + sub : a.T - 1;
    const float* row = a.logits + static_cast<size_t>(t) * a.E;
    __syncwarp();
    // the row, vectors or scores in turn to the lanes of the token
    float* slots = mem + sub * 8 * S;
    if (a.vecs) {
#pragma unroll
      for (int k = 0; k < LISTS; ++k) {
        const int e = (k * 8 + l) * 4;
        if (e < a.E) {
          const int to = full ? e / P : static_cast<int>((e * a.div_per) >> 20);
          copy16_async(slots + to * S + e - to * a.per, row + e);
        }
      }
    } else {
      for (int e = l; e < a.E; e += 8) {
        const int to = static_cast<int>((e * a.div_per) >> 20);
        slots[to * S + e - to * a.per] = load_global(row + e);
      }
    }
    copy_commit();
    copy_wait<0>();
    __syncwarp();
    float c[P];
#pragma unroll
    for (int k = 0; k < LISTS; ++k) {
      const float4 q = *reinterpret_cast<const float4*>(own + 4 * k);
      c[4 * k] = fmaxf(q.x, -INFINITY), c[4 * k + 1] = fmaxf(q.y, -INFINITY);
      c[4 * k + 2] = fmaxf(q.z, -INFINITY), c[4 * k + 3] = fmaxf(q.w, -INFINITY);
    }
    if (!full) {
#pragma unroll
      for (int k = 0; k < P; ++k) c[k] = k < mine ? c[k] : -INFINITY;
    }
    float top = -INFINITY, inv = 1.0f, total = 1.0f;
    auto soft = [&](float x) { return isinf(top) ? (x == top ? 1.0f : 0.0f) : ex2((x - top) * G_LOG2E); };
    auto score = [&](float x) {
      if constexpr (SOFT) return soft(x) * inv;
      else return rcp(1.0f + ex2(-x * G_LOG2E));
    };
    if (soft_row) {
#pragma unroll
      for (int k = 0; k < P; ++k) top = fmaxf(top, c[k]);
      top = O::maxf(top);
      total = 0.0f;
#pragma unroll
      for (int k = 0; k < P; ++k) total += soft(c[k]);
      total = O::sum(total);
      if (top == -INFINITY) total = static_cast<float>(a.E);  // (not the lanes' empty places)
      inv = rcp(total);
    }
    if constexpr (BIASED) {
#pragma unroll
      for (int k = 0; k < LISTS; ++k) {
        const float4 b = *reinterpret_cast<const float4*>(bias + l * (P + 4) + 4 * k);
        c[4 * k] = score(c[4 * k]) + b.x, c[4 * k + 1] = score(c[4 * k + 1]) + b.y;
        c[4 * k + 2] = score(c[4 * k + 2]) + b.z, c[4 * k + 3] = score(c[4 * k + 3]) + b.w;
      }
    }
    // (how far apart: as in group_gate_kernel)
    const float unsure = SOFT ? (BIASED ? 0x1p-16f : 0x1p-20f) * inv : 0x1p-20f;
    bool doubt = false, in = true;
    if (grouped) {
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        m2 = fmaxf(m2, fminf(m1, c[k]));
        m1 = fmaxf(m1, c[k]);
      }
      for (int o = lpg >> 1; o > 0; o >>= 1) {
        const float o1 = __shfl_xor_sync(0xFFFFFFFFu, m1, o), o2 = __shfl_xor_sync(0xFFFFFFFFu, m2, o);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      const float x1 = m1, x2 = m2;  // (logits without a bias)
      if (!two) m2 = 0.0f;
      else if (!BIASED) m1 = score(m1), m2 = score(m2);
      // lanes of groups before this one in the order
      const float rank = fmaxf(m1 + m2, -INFINITY);
      int before = 0;
#pragma unroll
      for (int d = 1; d < 8; ++d) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, rank, d);
        const int g = (l ^ d) >> a.log_lpg;
        before += g != group && (other > rank || (other == rank && g < group));
      }
      in = before < a.kept * lpg;
      if (BIASED || two) {
        const float big = (isinf(m1) ? 0.0f : fabsf(m1)) + (isinf(m2) ? 0.0f : fabsf(m2));
        const float last = -O::maxf(in ? -rank : -INFINITY), next = O::maxf(in ? -INFINITY : rank);
        const float room = 2.0f * unsure + 0x1p-21f * O::maxf(big);
        doubt = !ranks_apart(last, next, room);
        // Groups next to the border: as in group_gate_wide_kernel.
        const bool here = doubt && !(SOFT && isinf(top));
        if (__any_sync(0xFFFFFFFFu, here)) {
          const double sum = SOFT ? softmax_total64<8>(row, a.E, l, top) : 0.0;
          const bool near = here && (room == INFINITY || (in ? rank - next <= room : last - rank <= room));
          bool told = near;
          double exact;
          if constexpr (BIASED) {
            const float least = (two ? m2 : m1) - room;
            int count = 0, places = 0;
#pragma unroll
            for (int k = 0; k < P; ++k) {
              const bool one = near && (full || k < mine) && c[k] >= least;
              count += one;
              places = one ? places << 8 | k : places;
            }
            int all = count;
            for (int o = lpg >> 1; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
            told = near && all == (two ? 2 : 1);
            const int e = count > 0 ? l * a.per + (places & 255) : 0, f = count > 1 ? l * a.per + (places >> 8 & 255) : 0;
            const double2 d = biased_scores64<SOFT>(load_global(row + e), load_global(a.bias + e), load_global(row + f), load_global(a.bias + f), top, sum);
            exact = (count > 0 ? d.x : 0.0) + (count > 1 ? d.y : 0.0);
            for (int o = lpg >> 1; o > 0; o >>= 1) exact += __shfl_xor_sync(0xFFFFFFFFu, exact, o);
          } else {
            const double2 d = biased_scores64<SOFT>(x1, 0.0f, x2, 0.0f, top, sum);
            exact = d.x + d.y;
          }
          exact = told ? fmax(exact, static_cast<double>(-INFINITY)) : rank;
          int ahead = 0;  // lanes of groups
#pragma unroll
          for (int k = 1; k < 8; ++k) {
            const double other = __shfl_xor_sync(0xFFFFFFFFu, exact, k);
            const int g = (l ^ k) >> a.log_lpg;
            ahead += g != group && (other > exact || (other == exact && g < group));
          }
          if (O::any(near && !told) == 0u && here) {
            in = ahead < a.kept * lpg;
            doubt = false;
          }
        }
      }
    }
    // lists of four, largest first, equal ones in order
    float h[LISTS];
    int at[LISTS];
#pragma unroll
    for (int q = 0; q < LISTS; ++q) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = full || q * 4 + k < mine ? c[q * 4 + k] : NAN;
      uint32_t id[4] = {0, 1, 2, 3};
      auto sort2 = [&](int k) {  // neighbours, if out of order
        const bool swap = v[k] < v[k + 1];
        const float hi = swap ? v[k + 1] : v[k], lo = swap ? v[k] : v[k + 1];
        const uint32_t one = swap ? id[k + 1] : id[k], other = swap ? id[k] : id[k + 1];
        v[k] = hi, v[k + 1] = lo, id[k] = one, id[k + 1] = other;
      };
      sort2(0), sort2(1), sort2(2), sort2(0), sort2(1), sort2(0);
      float2* list = reinterpret_cast<float2*>(own + q * 6);
      list[0] = make_float2(v[0], v[1]);
      list[1] = make_float2(v[2], v[3]);
      list[2] = make_float2(NAN, __uint_as_float(id[0] | id[1] << 8 | id[2] << 16 | id[3] << 24));
      h[q] = in ? v[0] : NAN;
      at[q] = lane * S + q * 6;
    }
    auto head = [&] {
      float m = h[0];
#pragma unroll
      for (int q = 1; q < LISTS; ++q) m = fmaxf(m, h[q]);
      return O::maxf(m);
    };
    // the expert at a place of the lists
    auto expert = [&](int where) {
      const int rest = where - sub * 8 * S, of = rest / S, in_lane = rest - of * S, q = in_lane / 6;
      const uint32_t order = __float_as_uint(mem[(sub * 8 + of) * S + q * 6 + 5]);
      return of * a.per + q * 4 + static_cast<int>(order >> (in_lane - q * 6) * 8 & 3u);
    };
    float value = NAN;  // of the choice that this lane stands for
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= a.topk) break;
      const float best = head();
      value = l == j ? best : value;
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        if (h[q] == best) {
          pick[j] = at[q];
          h[q] = mem[++at[q]];
        }
      }
    }
    int taken = 0;
#pragma unroll
    for (int q = 0; q < LISTS; ++q) taken += at[q] - (lane * S + q * 6);
    taken += __shfl_xor_sync(0xFFFFFFFFu, taken, 1);
    taken += __shfl_xor_sync(0xFFFFFFFFu, taken, 2);
    taken += __shfl_xor_sync(0xFFFFFFFFu, taken, 4);
    if (__any_sync(0xFFFFFFFFu, taken != a.topk)) {
      // several lists had the largest: the rounds again, the first expert takes it
      __syncwarp();
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        at[q] = lane * S + q * 6;
        h[q] = in ? own[q * 6] : NAN;
      }
      for (int j = 0; j < a.topk; ++j) {
        const float best = head();
        value = l == j ? best : value;
        uint32_t of = 0xFFFFFFFFu;
#pragma unroll
        for (int q = LISTS - 1; q >= 0; --q)
          if (h[q] == best) of = expert(at[q]);
        const uint32_t e = O::min(of);
        bool here = of == e && of != 0xFFFFFFFFu;
#pragma unroll
        for (int q = 0; q < LISTS; ++q) {
          if (here && h[q] == best) {
            pick[j] = at[q];
            h[q] = mem[++at[q]];
            here = false;
          }
        }
      }
    }
    __syncwarp();
    const bool here = l < a.topk;
    int e = here ? expert(pick[l]) : 0;
    if constexpr (BIASED) {
      float next = h[0];
#pragma unroll
      for (int q = 1; q < LISTS; ++q) next = fmaxf(next, h[q]);
      next = O::maxf(next);  // the best one left, NaN if none is
      auto apart = [&](float hi, float lo) { return hi - lo > unsure + 0x1p-23f * (fabsf(hi) + fabsf(lo)); };
      auto same = [&](int f, int g) {
        return load_global(row + f) == load_global(row + g) && load_global(a.bias + f) == load_global(a.bias + g);
      };
      const float after = __shfl_down_sync(0xFFFFFFFFu, value, 1, 8), lo = l + 1 < a.topk ? after : next;
      const bool close = here && lo == lo && !apart(value, lo);
      const int follower = __shfl_down_sync(0xFFFFFFFFu, e, 1, 8);
      const float end = __shfl_sync(0xFFFFFFFFu, value, a.topk - 1, 8);
      const int last = __shfl_sync(0xFFFFFFFFu, e, a.topk - 1, 8);
      if (__any_sync(0xFFFFFFFFu, close)) {
        // equal inputs have equal values: their order is that of the indexes
        bool unsorted = close && l + 1 < a.topk && !same(e, follower);
        // and what was left out next to the last one in
        uint32_t out = 0xFFFFFFFFu, others = 0, equal = 0;
#pragma unroll
        for (int q = 0; q < LISTS; ++q) {
          for (int i = in ? at[q] : lane * S + q * 6 + 4; i < lane * S + q * 6 + 4; ++i) {
            if (mem[i] != mem[i] || apart(end, mem[i])) continue;
            const int f = expert(i);
            if (same(last, f)) {
              ++equal;
            } else {
              ++others;
              out = f;
            }
          }
        }
        others = static_cast<uint32_t>(O::sum(static_cast<float>(others)));
        out = O::min(out);
        equal = O::any(equal);
        unsorted = O::any(unsorted || others > 0u) != 0u;
        const bool full_choice = (SOFT && isinf(top)) || others > 1u || equal != 0u;
        if (full_choice) doubt |= unsorted;
        // Mostly it is two neighbours, or the last one in and the first one out: their order
        // is told by the doubles of these nine alone.
        const bool nine = unsorted && !full_choice;
        if (__any_sync(0xFFFFFFFFu, nine)) {
          const int f = others == 1u ? static_cast<int>(out) : -1;
          const double sum = SOFT ? softmax_total64<8>(row, a.E, l, top) : 0.0;
          const int2 place = order64<8, SOFT>(row, a.bias, e, f, l, a.topk, top, sum);
          __syncwarp();
          if (nine && here && place.x < a.topk) pick[place.x] = e;
          if (nine && l == 0 && f >= 0 && place.y < a.topk) pick[place.y] = f;
          __syncwarp();
          if (nine && here) e = pick[l];
        }
      }
    }
    uint32_t doubts = __ballot_sync(0xFFFFFFFFu, doubt);
    while (doubts != 0u) {  // token by token, by the whole warp
      const int of = (__ffs(doubts) - 1) >> 3;
      doubts &= ~(0xFFu << of * 8);
      const long long u = __shfl_sync(0xFFFFFFFFu, t, of * 8);
      __syncwarp();
      choose64<32>(a, a.logits + static_cast<size_t>(u) * a.E, kept64, pick64, lane, 0xFFFFFFFFu);
      if (sub == of && here) e = expert_at(a, kept64, pick64[l]);
      __syncwarp();
    }
    // the weights, with the rules of group_gate_kernel
    const float x = here ? fmaxf(load_global(row + e), -INFINITY) : -INFINITY;
    const float peak = a.renorm ? O::maxf(x) : 0.0f;
    float w;
    if constexpr (SOFT) {
      const float from = a.renorm ? peak : top;
      w = isinf(from) ? (x == from ? 1.0f : 0.0f) : expf(x - from);
    } else {
      w = !a.renorm || peak > -64.0f ? rcp(1.0f + expf(-x)) : peak == -INFINITY ? 1.0f : expf(x - peak);
    }
    w = here ? w : 0.0f;
    const float sum = a.renorm ? O::sum(w) : total;
    if (here && token) {
      a.ids[static_cast<size_t>(t) * a.topk + l] = e;
      a.weights[static_cast<size_t>(t) * a.topk + l] = a.scale * w * rcp(sum);
    }
  }
}

// Gradient of the scores where only the chosen ones have one (sigmoid, or weights
// that are renormalised).  A token's slots lie in SLOTS neighbouring lanes, so that a
// warp works on 32 / SLOTS tokens at once; it writes their rows, which lie behind one
// another, with zeros, and then the slots' gradients over them.  Bound by memory: 131072
// x 256 34 us for 134 MB written and 75 MB read (a chosen score brings its sector of 32
// bytes).
template <int SLOTS>
__global__ void __launch_bounds__(GG_THREADS)
group_gate_bwd_chosen_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int TPW = 32 / SLOTS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % SLOTS;
  auto sum = [](float v) {
#pragma unroll
    for (int o = SLOTS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  auto largest = [](float v) {
#pragma unroll
    for (int o = SLOTS / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  };
  wait_for_previous();
  for (long long t0 = (static_cast<long long>(blockIdx.x) * GG_WARPS + warp) * TPW; t0 < a.T; t0 += static_cast<long long>(gridDim.x) * GG_WARPS * TPW) {
    const long long t = t0 + lane / SLOTS;
    const int tokens = static_cast<int>(min(static_cast<long long>(TPW), a.T - t0));
    int id = -1;
    float g = 0.0f, x = -INFINITY;
    if (t < a.T && l < a.topk) {
      id = load_global(a.ids_in + t * a.topk + l);
      if (id >= a.E) id = -1;
      g = a.scale * load_global(a.dweights + t * a.topk + l);
      if (id >= 0) x = fmaxf(load_global(a.logits + t * a.E + id), -INFINITY);
    }
    if (!a.accumulate) {
      float* rows = a.dlogits + t0 * a.E;
      const int n = tokens * a.E;
      if (a.E % 4 == 0 || TPW % 4 == 0) {  // rows begin on 16 bytes
        for (int i = lane * 4; i + 3 < n; i += 128) *reinterpret_cast<float4*>(rows + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (lane < n % 4) rows[n - n % 4 + lane] = 0.0f;
      } else {
        for (int i = lane; i < n; i += 32) rows[i] = 0.0f;
      }
      __syncwarp();  // the gradients come over the zeros
    }
    // the weights, as the forward pass has them
    float d;
    const float small = expf(-fabsf(x)), left = (x > 0.0f ? small : 1.0f) / (1.0f + small);  // 1 - sigmoid
    if (a.renorm) {
      const float peak = largest(x);
      const bool constant = a.softmax ? isinf(peak) : peak == -INFINITY;  // no weight depends on a score
      float v = 0.0f;
      if (id >= 0 && !constant) v = a.softmax ? expf(x - peak) : expf(fminf(x, 0.0f) - fminf(peak, 0.0f)) / (1.0f + small);
      const float total = sum(v), dot = sum(v * g) / total;
      d = constant ? 0.0f : v / total * (g - dot) * (a.softmax ? 1.0f : left);
    } else {
      d = (x > 0.0f ? 1.0f : small) / (1.0f + small) * left * g;
    }
    if (id >= 0) {
      float* at = a.dlogits + t * a.E + id;
      *at = a.accumulate ? *at + d : d;
    }
  }
}

constexpr int bwd_ctas(int v) { return v <= 2 ? 6 : v == 4 ? 4 : 3; }  // per SM

// The same for tokens of more than 32 slots, and the softmax that is not renormalised:
// every score has a gradient, -p sum_i p_i g_i, and the chosen ones p g more.  LPT lanes
// hold a token's scores in V vectors of four (or, for rows that do not begin on 16
// bytes, scores one by one).  A grid of as many CTAs as are on the GPU at once: 131072 x
// 256 57 us, with a sixth CTA where five fit an SM 98; 16 lanes a token, with 32 63 us
// (128 experts 35 and 53).
template <int LPT, int V>
__global__ void __launch_bounds__(GG_THREADS, bwd_ctas(V))
group_gate_bwd_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int TPW = 32 / LPT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPT;
  using O = Over<LPT>;
  const bool every = a.softmax && !a.renorm, vec = a.E % 4 == 0;
  wait_for_previous();
  for (long long t0 = (static_cast<long long>(blockIdx.x) * GG_WARPS + warp) * TPW; t0 < a.T; t0 += static_cast<long long>(gridDim.x) * GG_WARPS * TPW) {
    const bool here = t0 + lane / LPT < a.T;
    const size_t t = static_cast<size_t>(here ? t0 + lane / LPT : a.T - 1);
    const float* row = a.logits + t * a.E;
    float* out = a.dlogits + t * a.E;
    auto expert = [&](int v, int i) { return vec ? (v * LPT + l) * 4 + i : (v * 4 + i) * LPT + l; };
    struct Slot {
      int e;
      float g, x;
    };
    auto load = [&](int j) {
      const int e = load_global(a.ids_in + t * a.topk + j);
      const float g = a.scale * load_global(a.dweights + t * a.topk + j);
      return Slot{e < a.E ? e : -1, g, e >= 0 && e < a.E ? fmaxf(load_global(row + e), -INFINITY) : -INFINITY};
    };
    // a lane's first slot is on its way before the row is worked on
    const Slot first = l < a.topk ? load(l) : Slot{-1, 0.0f, -INFINITY};
    auto slot = [&](int j) { return j == l ? first : load(j); };
    float f[V][4] = {};
    float peak = -INFINITY, total = 0.0f, dot = 0.0f;
    if (every) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (vec) {
          const int e = expert(v, 0);
          const float4 q = e < a.E ? load_global(reinterpret_cast<const float4*>(row + e)) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          f[v][0] = q.x, f[v][1] = q.y, f[v][2] = q.z, f[v][3] = q.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[v][i] = expert(v, i) < a.E ? load_global(row + expert(v, i)) : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) peak = fmaxf(peak, f[v][i] = fmaxf(f[v][i], -INFINITY));
      }
      peak = O::maxf(peak);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) total += f[v][i] = isinf(peak) ? 0.0f : ex2((f[v][i] - peak) * G_LOG2E);
      total = O::sum(total);
    } else if (a.renorm) {
      for (int j = l; j < a.topk; j += LPT) peak = fmaxf(peak, slot(j).x);
      peak = O::maxf(peak);
    }
    const bool constant = (every || a.renorm) && (a.softmax ? isinf(peak) : peak == -INFINITY);
    auto part = [&](float x) {  // of a chosen score, before the sum
      if (constant || x == -INFINITY) return 0.0f;
      if (a.softmax) return every ? ex2((x - peak) * G_LOG2E) : expf(x - peak);
      return expf(fminf(x, 0.0f) - (a.renorm ? fminf(peak, 0.0f) : 0.0f)) / (1.0f + expf(-fabsf(x)));
    };
    if (every || a.renorm) {
      float sum = 0.0f;
      for (int j = l; j < a.topk; j += LPT) {
        const Slot c = slot(j);
        const float v = part(c.x);
        sum += v;
        dot += v * c.g;
      }
      if (!every) total = O::sum(sum);
      dot = O::sum(dot);
      dot = constant ? 0.0f : dot / total;
    } else {
      total = 1.0f;
    }
    const float inv = constant ? 0.0f : 1.0f / total;
    // the rows without the chosen ones' own terms
    if (!a.accumulate || every) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float4 q = make_float4(-f[v][0] * inv * dot, -f[v][1] * inv * dot, -f[v][2] * inv * dot, -f[v][3] * inv * dot);
        if (!every) q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int e = expert(v, 0);
        if (vec) {
          if (here && e < a.E) {
            if (a.accumulate) {
              const float4 o = *reinterpret_cast<const float4*>(out + e);
              q.x += o.x, q.y += o.y, q.z += o.z, q.w += o.w;
            }
            *reinterpret_cast<float4*>(out + e) = q;
          }
        } else {
          const float s[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (here && expert(v, i) < a.E) out[expert(v, i)] = a.accumulate ? out[expert(v, i)] + s[i] : s[i];
        }
      }
      __syncwarp();
    }
    for (int j = l; j < a.topk; j += LPT) {
      const Slot c = slot(j);
      const int e = c.e;
      if (e < 0 || !here) continue;
      const float x = c.x, g = c.g, p = part(x) * inv;
      float d = a.renorm || every ? p * (g - dot) : p * g;
      if (!a.softmax) {
        const float small = expf(-fabsf(x));
        d *= (x > 0.0f ? small : 1.0f) / (1.0f + small);
      }
      // over the zero or the row's term; with accumulate onto what was there, of which
      // the row's term is a part by now
      out[e] = !a.accumulate ? d : out[e] + (every ? p * g : d);
    }
  }
}

flux_status_t check_gate(int T, int E, int topk, int score, float scale, const float* logits) {
  if (T < 0 || E < 1 || E > FLUX_MAX_EXPERTS || topk < 1 || topk > E) return FLUX_ERR_INVALID_ARG;
  if (score != FLUX_SCORE_SOFTMAX && score != FLUX_SCORE_SIGMOID) return FLUX_ERR_INVALID_ARG;
  if (!isfinite(scale)) return FLUX_ERR_INVALID_ARG;
  if (T > 0 && logits == nullptr) return FLUX_ERR_INVALID_ARG;
  return aligned16(logits) ? FLUX_OK : FLUX_ERR_UNSUPPORTED;
}

template <int NC>
flux_status_t launch_gate(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int TPC = GG_WARPS * 4;
  constexpr auto kernel = group_gate_kernel<NC>;
  const size_t smem = TPC * gate_token_bytes(a.row, a.topk);
  static OncePerDevice once;
  const cudaError_t attr = once(dev.device, [&dev] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dev.max_smem_optin));
  });
  if (attr != cudaSuccess) return cuda_fail(attr);
  const int per_sm = static_cast<int>(std::max<size_t>(1, std::min<size_t>(5, (227u << 10) / (smem + 1024))));
  const int grid = std::min(ceil_div(a.T, TPC), GG_SMS * per_sm);
  const cudaError_t e = launch_behind(kernel, dim3(grid), GG_THREADS, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int VECS, int LISTS, bool GROUPED, bool SOFT, bool BIASED>
flux_status_t launch_wide(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr auto kernel = group_gate_wide_kernel<VECS, LISTS, GROUPED, SOFT, BIASED>;
  const size_t smem = sizeof(float) * (GG_WARPS * wide_words(a.vecs, a.row, a.topk, LISTS) + (BIASED ? 128 * a.vecs : 0));
  static OncePerDevice once;
  const cudaError_t attr = once(dev.device, [&dev] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dev.max_smem_optin));
  });
  if (attr != cudaSuccess) return cuda_fail(attr);
  const int per_sm = static_cast<int>(std::max<size_t>(1, std::min<size_t>(LISTS <= 2 ? 4 : 3, (227u << 10) / (smem + 1024))));
  const int grid = std::min(ceil_div(a.T, GG_WARPS), GG_SMS * per_sm);
  const cudaError_t e = launch_behind(kernel, dim3(grid), GG_THREADS, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int VECS, int LISTS, bool GROUPED>
flux_status_t launch_wide(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.softmax) return a.bias ? launch_wide<VECS, LISTS, GROUPED, true, true>(a, dev, s) : launch_wide<VECS, LISTS, GROUPED, true, false>(a, dev, s);
  return a.bias ? launch_wide<VECS, LISTS, GROUPED, false, true>(a, dev, s) : launch_wide<VECS, LISTS, GROUPED, false, false>(a, dev, s);
}

// Rows of up to 256 experts have their loops unrolled.
template <bool GROUPED>
flux_status_t launch_wide(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const int lists = ceil_div(a.kept * a.np, 128);
  if (a.vecs == 1) return launch_wide<1, 1, GROUPED>(a, dev, s);
  if (a.vecs == 2 && lists == 2) return launch_wide<2, 2, GROUPED>(a, dev, s);
  if constexpr (GROUPED) {
    if (a.vecs == 2) return launch_wide<2, 1, true>(a, dev, s);
    if (lists == 1) return launch_wide<0, 1, true>(a, dev, s);
    if (lists == 2) return launch_wide<0, 2, true>(a, dev, s);
  }
  if (lists <= 4) return launch_wide<0, 4, GROUPED>(a, dev, s);
  if (lists <= 8) return launch_wide<0, 8, GROUPED>(a, dev, s);
  return launch_wide<0, 9, GROUPED>(a, dev, s);  // more than 1024 places
}

template <int P, bool SOFT, bool BIASED>
flux_status_t launch_octet(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr auto kernel = group_gate_octet_kernel<P, SOFT, BIASED>;
  constexpr int PER_SM = P == 32 ? 3 : 4;
  const int smem = static_cast<int>(sizeof(float)) * (GG_WARPS * octet_words(octet_pitch<P>()) + (BIASED ? 8 * (P + 4) : 0));
  static OncePerDevice once;
  const cudaError_t attr = once(dev.device, [smem] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (attr != cudaSuccess) return cuda_fail(attr);
  const int grid = std::min(ceil_div(a.T, GG_WARPS * 4), GG_SMS * PER_SM);
  const cudaError_t e = launch_behind(kernel, dim3(grid), GG_THREADS, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int P>
flux_status_t launch_octet(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.softmax) return a.bias ? launch_octet<P, true, true>(a, dev, s) : launch_octet<P, true, false>(a, dev, s);
  return a.bias ? launch_octet<P, false, true>(a, dev, s) : launch_octet<P, false, false>(a, dev, s);
}

template <int SLOTS>
flux_status_t launch_bwd_chosen(const GroupGateArgs& a, cudaStream_t s) {
  const int grid = std::min(ceil_div(a.T, GG_WARPS * (32 / SLOTS)), GG_SMS * 8);
  const cudaError_t e = launch_behind(group_gate_bwd_chosen_kernel<SLOTS>, dim3(grid), GG_THREADS, 0, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int LPT, int V>
flux_status_t launch_bwd(const GroupGateArgs& a, cudaStream_t s) {
  const int grid = std::min(ceil_div(a.T, GG_WARPS * (32 / LPT)), GG_SMS * bwd_ctas(V));
  const cudaError_t e = launch_behind(group_gate_bwd_kernel<LPT, V>, dim3(grid), GG_THREADS, 0, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

flux_status_t launch_gate_bwd(const GroupGateArgs& a, cudaStream_t s) {
  if (!(a.softmax && !a.renorm) && a.topk <= 32) {
    if (a.topk <= 2) return launch_bwd_chosen<2>(a, s);
    if (a.topk <= 4) return launch_bwd_chosen<4>(a, s);
    if (a.topk <= 8) return launch_bwd_chosen<8>(a, s);
    return launch_bwd_chosen<32>(a, s);
  }
  if (a.E <= 32) return launch_bwd<8, 1>(a, s);
  if (a.E <= 64) return launch_bwd<8, 2>(a, s);
  if (a.E <= 128) return launch_bwd<16, 2>(a, s);
  if (a.E <= 256) return launch_bwd<16, 4>(a, s);
  if (a.E <= 512) return launch_bwd<32, 4>(a, s);
  return launch_bwd<32, 8>(a, s);
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" flux_status_t flux_moe_group_gate(int T, int E, int topk, int score, int groups, int topk_groups,
                                             int group_top, int renorm, float scale, const float* logits,
                                             const float* bias, int32_t* topk_ids, float* topk_weights,
                                             void* stream) {
  flux_status_t st = check_gate(T, E, topk, score, scale, logits);
  if (st == FLUX_ERR_INVALID_ARG) return st;
  if (groups < 1 || groups > FLUX_MAX_GROUPS || E % groups != 0 || topk_groups < 1 || topk_groups > groups ||
      topk > topk_groups * (E / groups) || group_top < 1 || group_top > 2)
    return FLUX_ERR_INVALID_ARG;
  if (T > 0 && (topk_ids == nullptr || topk_weights == nullptr)) return FLUX_ERR_INVALID_ARG;
  if (st != FLUX_OK) return st;
  if (!aligned16(bias) || !aligned16(topk_ids) || !aligned16(topk_weights)) return FLUX_ERR_UNSUPPORTED;
  if (T == 0) return FLUX_OK;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  GroupGateArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.T = T;
  a.E = E;
  a.topk = topk;
  a.G = topk_groups < groups ? groups : 1;  // where all are kept there might as well be one
  a.kept = topk_groups < groups ? topk_groups : 1;
  a.top = group_top;
  a.n = E / a.G;
  a.div_n = ((1u << 20) + a.n - 1) / a.n;
  a.softmax = score == FLUX_SCORE_SOFTMAX;
  a.renorm = renorm != 0;
  a.scale = scale;
  // Eight lanes a token where its groups fit them
  const bool grouped = topk_groups < groups;
  const int lanes = !grouped ? 8 : groups <= 8 && 8 % groups == 0 ? 8 / groups : 0;  // of a group
  // A warp a token is faster while a warp has at most two or three of them (256 experts, 8
  // groups, us with cold caches, a warp a token and eight lanes: 13 tokens 4.1 and 6.2,
  // 4864 10 and 14, 9728 13 and 16, 19456 20 and 20, 131072 120 and 80).
  const bool lone = T <= 64 * GG_SMS && E > 64;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (topk <= 8 && E <= 256 && !lone && lanes > 0 && (!grouped || a.n % lanes == 0)) {
    a.per = grouped ? a.n / lanes : ceil_div(E, 8);
    a.div_per = ((1u << 20) + a.per - 1) / a.per;
    while (grouped && 1 << a.log_lpg < lanes) ++a.log_lpg;
    a.vecs = a.per % 4 == 0 && E % 4 == 0;
    if (a.per <= 4) return launch_octet<4>(a, dev, s);
    if (a.per <= 8) return launch_octet<8>(a, dev, s);
    if (a.per <= 16) return launch_octet<16>(a, dev, s);
    return launch_octet<32>(a, dev, s);
  }
  const bool wide = E > 64 || T <= 64 * GG_SMS;
  const int lpt = wide ? 32 : 8;
  a.lpg = lpt;  // lanes of a group: as many as let all groups be ranked at once, at least one
  while (a.lpg > 1 && a.lpg * a.G > lpt) a.lpg /= 2;
  while (1 << a.log_lpg < a.lpg) ++a.log_lpg;
  if (!wide) {
    // (pad: words between the groups' rows, so that lanes of neighbouring groups read other banks)
    a.pad = grouped ? a.lpg : 0;
    a.row = E + a.G * a.pad;
    const int each = ceil_div(a.kept * a.n, lpt);  // candidates of a lane
    if (each <= 1) return launch_gate<1>(a, dev, s);
    if (each <= 2) return launch_gate<2>(a, dev, s);
    if (each <= 4) return launch_gate<4>(a, dev, s);
    return launch_gate<8>(a, dev, s);
  }
  a.np = (a.n + 3) / 4 * 4;
  a.div_np = ((1u << 20) + a.np - 1) / a.np;
  a.pad = !grouped || a.lpg >= 8 ? 0 : (4 * a.lpg - a.np % 32 + 32) % 32;
  a.vecs = ceil_div(a.G * a.np, 128);
  a.trips = ceil_div(a.np, 4 * a.lpg);
  a.rivals = ceil_div(a.G, a.lpg);
  a.row = !grouped ? 0 : 128 * a.vecs + (128 * a.vecs - 4) / a.np * a.pad;  // values of every place
  return grouped ? launch_wide<true>(a, dev, s) : launch_wide<false>(a, dev, s);
}

extern "C" flux_status_t flux_moe_group_gate_bwd(int T, int E, int topk, int score, int renorm, float scale,
                                                 const float* logits, const int32_t* topk_ids,
                                                 const float* dweights, int accumulate, float* dlogits,
                                                 void* stream) {
  flux_status_t st = check_gate(T, E, topk, score, scale, logits);
  if (st == FLUX_ERR_INVALID_ARG) return st;
  if (T > 0 && (topk_ids == nullptr || dweights == nullptr || dlogits == nullptr)) return FLUX_ERR_INVALID_ARG;
  if (st != FLUX_OK) return st;
  if (!aligned16(topk_ids) || !aligned16(dweights) || !aligned16(dlogits)) return FLUX_ERR_UNSUPPORTED;
  if (T == 0) return FLUX_OK;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  GroupGateArgs a{};
  a.logits = logits;
  a.ids_in = topk_ids;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.T = T;
  a.E = E;
  a.topk = topk;
  a.softmax = score == FLUX_SCORE_SOFTMAX;
  a.renorm = renorm != 0;
  a.accumulate = accumulate != 0;
  a.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_gate_bwd(a, s);
}
