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
  int lpg;             // lanes that rank one group
  uint32_t div_n;      // ceil(2^20 / n): e / n = e div_n >> 20 for e < 1024
  int row;             // values of a token's row in shared memory
  int softmax, renorm, accumulate;
  float scale;
};

// What a token needs in shared memory: its values (room for doubles), the picked
// experts, the groups' ranks, the ranks in order, the kept groups.
__host__ __device__ inline size_t gate_token_bytes(int row, int topk) {
  return static_cast<size_t>(row) * 8 + ((topk * 4 + 7) & ~7) + 32 * 8 * 2 + 32 * 4;
}

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

// f(e, logit) for the lane's experts of a row, a NaN as -inf.
template <int LPT, typename F>
__device__ __forceinline__ void each_logit(const float* row, int E, int l, F&& f) {
  if (E % 4 == 0) {
#pragma unroll 2
    for (int e = l * 4; e < E; e += LPT * 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(row + e));
      f(e, fmaxf(q.x, -INFINITY));
      f(e + 1, fmaxf(q.y, -INFINITY));
      f(e + 2, fmaxf(q.z, -INFINITY));
      f(e + 3, fmaxf(q.w, -INFINITY));
    }
  } else {
#pragma unroll 4
    for (int e = l; e < E; e += LPT) f(e, fmaxf(__ldg(row + e), -INFINITY));
  }
}

// A token's places in shared memory.
struct Rows {
  float* val;
  double* val64;
  int32_t* pick;
  float *rank, *sorted;
  double *rank64;
  int32_t* kept;
  __device__ __forceinline__ Rows(char* base, int row, int topk) {
    val64 = reinterpret_cast<double*>(base);
    val = reinterpret_cast<float*>(base);
    pick = reinterpret_cast<int32_t*>(base + static_cast<size_t>(row) * 8);
    rank64 = reinterpret_cast<double*>(base + static_cast<size_t>(row) * 8 + ((topk * 4 + 7) & ~7));
    rank = reinterpret_cast<float*>(rank64);
    sorted = rank + 32;
    kept = reinterpret_cast<int32_t*>(rank64 + 64);
  }
};

__device__ __forceinline__ int group_of(const GroupGateArgs& a, int e) { return static_cast<int>((e * a.div_n) >> 20); }
__device__ __forceinline__ int place(const GroupGateArgs& a, int e) { return a.pad == 0 ? e : e + group_of(a, e) * a.pad; }
// The expert at place p of the kept groups' experts in order.
__device__ __forceinline__ int expert_at(const GroupGateArgs& a, const Rows& r, int p) {
  if (a.kept == a.G) return p;
  const int q = group_of(a, p);
  return r.kept[q] * a.n + (p - q * a.n);
}

// The choice in doubles, by the LPT lanes of one token (mask).  Rare.
template <int LPT, int NC>
__device__ __noinline__ void choose64(const GroupGateArgs& a, const float* row, const Rows& r, int l, uint32_t mask) {
  auto shfl = [&](double v, int o) { return __shfl_xor_sync(mask, v, o); };
  auto logit = [&](int e) {
    const float x = __ldg(row + e);
    return static_cast<double>(x != x ? -INFINITY : x);
  };
  double top = -INFINITY, total = 0.0;
  if (a.softmax) {
    for (int e = l; e < a.E; e += LPT) top = fmax(top, logit(e));
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) top = fmax(top, shfl(top, o));
    for (int e = l; e < a.E; e += LPT) total += isinf(top) ? (logit(e) == top ? 1.0 : 0.0) : exp(logit(e) - top);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) total += shfl(total, o);
  }
  auto score = [&](double x) {
    if (!a.softmax) return 1.0 / (1.0 + exp(-x));
    return (isinf(top) ? (x == top ? 1.0 : 0.0) : exp(x - top)) / total;
  };
  __syncwarp(mask);
  for (int e = l; e < a.E; e += LPT) {
    const double x = logit(e), c = a.bias != nullptr ? score(x) + static_cast<double>(__ldg(a.bias + e)) : x;
    r.val64[place(a, e)] = c != c ? -INFINITY : c;
  }
  __syncwarp(mask);
  if (a.kept < a.G) {
    double mine[32 / LPT];
    for (int g = l, i = 0; g < a.G; g += LPT, ++i) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int m = 0; m < a.n; ++m) {
        const double v = r.val64[g * (a.n + a.pad) + m];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
      if (a.top == 2 && a.n > 1) m1 = a.bias != nullptr ? m1 + m2 : score(m1) + score(m2);
      r.rank64[g] = m1 != m1 ? -INFINITY : m1;
    }
    __syncwarp(mask);
    for (int g = l, i = 0; g < a.G; g += LPT, ++i) mine[i] = r.rank64[g];
    uint32_t in = 0;
    for (int g = l, i = 0; g < a.G; g += LPT, ++i) {
      int pos = 0;
      for (int o = 0; o < a.G; ++o) pos += r.rank64[o] > mine[i] || (r.rank64[o] == mine[i] && o < g);
      if (pos < a.kept) in |= 1u << g;
    }
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) in |= __shfl_xor_sync(mask, in, o);
    __syncwarp(mask);
    for (int g = l; g < a.G; g += LPT)
      if (in >> g & 1u) r.kept[__popc(in & ((1u << g) - 1u))] = g;
    __syncwarp(mask);
  }
  const int count = a.kept * a.n;
  uint32_t taken = 0;
  for (int j = 0; j < a.topk; ++j) {
    double best = -INFINITY;
    int at = 1 << 20;
    for (int i = 0; i < NC; ++i) {
      const int p = i * LPT + l;
      if (p >= count || (taken >> i & 1u)) continue;
      const int e = expert_at(a, r, p);
      const double v = r.val64[place(a, e)];
      if (at == 1 << 20 || v > best) {
        best = v;
        at = p;
      }
    }
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) {
      const double ov = shfl(best, o);
      const int oat = __shfl_xor_sync(mask, at, o);
      if (oat != 1 << 20 && (at == 1 << 20 || ov > best || (ov == best && oat < at))) {
        best = ov;
        at = oat;
      }
    }
    if (at % LPT == l) taken |= 1u << at / LPT;
    if (l == 0) r.pick[j] = expert_at(a, r, at);
  }
  __syncwarp(mask);
}

// One token to LPT lanes, NC candidates each.  The lanes put the values into a row
// of shared memory, rank the groups from there, and take their candidates (those
// of the kept groups, in order) into registers for topk rounds of a maximum.
template <int LPT, int NC>
__global__ void __launch_bounds__(GG_THREADS, NC <= 8 ? 5 : 2)
group_gate_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int TPW = 32 / LPT;
  extern __shared__ double smem[];
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
          r.val[at] = fmaxf(r.val[at] * inv + __ldg(a.bias + e), -INFINITY);
        };
        if (a.E % 4 == 0) {
          for (int e = l * 4; e < a.E; e += LPT * 4) third(e), third(e + 1), third(e + 2), third(e + 3);
        } else {
          for (int e = l; e < a.E; e += LPT) third(e);
        }
      }
    } else {
      each_logit<LPT>(row, a.E, l, [&](int e, float x) {
        r.val[place(a, e)] = biased ? fmaxf(score(x) + __ldg(a.bias + e), -INFINITY) : x;
      });
    }
    __syncwarp();
    // How far apart two values have to be for their order to be sure: errors of the
    // sigmoid 4.4 2^-24 (argument, ex2, sum, reciprocal), of the softmax 70 2^-24 of its
    // largest, and half an ulp for the bias; twice that for two values, and a margin.
    const float unsure = a.softmax ? 0x1p-16f * inv : 0x1p-20f;
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
        doubt = !(r.sorted[a.kept - 1] - r.sorted[a.kept] > 2.0f * unsure + 0x1p-21f * big);
    }
    const int count = a.kept * a.n;
    uint32_t key[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = i * LPT + l;
      key[i] = p < count ? order_of(r.val[place(a, expert_at(a, r, p))]) : 0u;
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
      if (l == 0) r.pick[j] = expert_at(a, r, static_cast<int>(at));
    }
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NC; ++i) m = max(m, key[i]);
    m = O::max(m);  // the best one left, 0 if none is
    __syncwarp();
    if (biased) {
      auto apart = [&](float hi, float lo) { return hi - lo > unsure + 0x1p-23f * (fabsf(hi) + fabsf(lo)); };
      auto same = [&](int e, int f) { return __ldg(row + e) == __ldg(row + f) && __ldg(a.bias + e) == __ldg(a.bias + f); };
      const float last = r.val[place(a, r.pick[a.topk - 1])];
      uint32_t close = m != 0u && !apart(last, value_of(m));
      for (int j = l; j + 1 < a.topk; j += LPT) close |= !apart(r.val[place(a, r.pick[j])], r.val[place(a, r.pick[j + 1])]);
      if (O::any(close)) {
        // equal inputs have equal values: their order is that of the indexes
        uint32_t wrong = 0;
        for (int j = l; j + 1 < a.topk; j += LPT) {
          const int e = r.pick[j], f = r.pick[j + 1];
          wrong |= !apart(r.val[place(a, e)], r.val[place(a, f)]) && !same(e, f);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (key[i] != 0u && !apart(last, value_of(key[i])))
            wrong |= !same(r.pick[a.topk - 1], expert_at(a, r, i * LPT + l));
        doubt |= wrong;
      }
    }
    doubt = O::any(doubt);
    if (doubt) choose64<LPT, NC>(a, row, r, l, LPT == 32 ? 0xFFFFFFFFu : ((1u << LPT % 32) - 1u) << (sub * LPT));
    __syncwarp();
    // the weights
    auto chosen = [&](int j) { return fmaxf(__ldg(row + r.pick[j]), -INFINITY); };
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
        a.ids[t * a.topk + j] = r.pick[j];
        a.weights[t * a.topk + j] = a.scale * (weight(chosen(j)) / sum);
      }
    }
  }
}

// Gradient of the scores.  The row of a token is made in shared memory (zeros but
// for the chosen experts, or the whole softmax) and written once.
template <int LPT>
__global__ void __launch_bounds__(GG_THREADS, 4)
group_gate_bwd_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int TPW = 32 / LPT;
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPT, sub = lane / LPT;
  using O = Over<LPT>;
  const int pitch = (a.E + 3) & ~3;
  float* out = reinterpret_cast<float*>(smem) + (warp * TPW + sub) * pitch;
  const bool every = a.softmax && !a.renorm;
  const bool sparse = a.accumulate && !every;  // only the chosen experts' gradients change
  wait_for_previous();
  for (int e = l; e < a.E; e += LPT) out[e] = 0.0f;
  for (long long t0 = static_cast<long long>(blockIdx.x * GG_WARPS + warp) * TPW; t0 < a.T; t0 += static_cast<long long>(gridDim.x) * GG_WARPS * TPW) {
    const bool here = t0 + sub < a.T;
    const size_t t = static_cast<size_t>(here ? t0 + sub : a.T - 1);
    const float* row = a.logits + t * a.E;
    const int32_t* ids = a.ids_in + t * a.topk;
    const float* dw = a.dweights + t * a.topk;
    auto inside = [&](int j) { return ids[j] >= 0 && ids[j] < a.E; };
    auto chosen = [&](int j) { return inside(j) ? fmaxf(__ldg(row + ids[j]), -INFINITY) : -INFINITY; };
    __syncwarp();
    if (every) {
      float top = -INFINITY, total = 0.0f;
      each_logit<LPT>(row, a.E, l, [&](int e, float x) {
        out[e] = x;
        top = fmaxf(top, x);
      });
      top = O::maxf(top);
      __syncwarp();
      for (int e = l; e < a.E; e += LPT) {
        out[e] = isinf(top) ? 0.0f : ex2((out[e] - top) * G_LOG2E);
        total += out[e];
      }
      total = O::sum(total);
      const float inv = isinf(top) ? 0.0f : 1.0f / total;
      __syncwarp();
      float dot = 0.0f;
      for (int j = l; j < a.topk; j += LPT)
        if (inside(j)) dot += out[ids[j]] * inv * (a.scale * __ldg(dw + j));
      dot = O::sum(dot);
      __syncwarp();
      // the sum's terms, then the chosen ones' own
      for (int e = l; e < a.E; e += LPT) out[e] *= -dot * inv;
      __syncwarp();
      for (int j = l; j < a.topk; j += LPT)
        if (inside(j) && !isinf(top)) out[ids[j]] += ex2((chosen(j) - top) * G_LOG2E) * inv * (a.scale * __ldg(dw + j));
    } else {
      float peak = -INFINITY, sum = 1.0f, dot = 0.0f;
      if (a.renorm) {
        for (int j = l; j < a.topk; j += LPT) peak = fmaxf(peak, chosen(j));
        peak = O::maxf(peak);
      }
      const bool constant = a.renorm && (a.softmax ? isinf(peak) : peak == -INFINITY);  // the weights do not depend on the scores
      auto part = [&](float x) {
        if (a.softmax) return expf(x - peak);
        return expf(fminf(x, 0.0f) - (a.renorm ? fminf(peak, 0.0f) : 0.0f)) / (1.0f + expf(-fabsf(x)));
      };
      if (a.renorm) {
        sum = 0.0f;
        for (int j = l; j < a.topk; j += LPT) {
          const float v = constant ? 0.0f : part(chosen(j));
          sum += v;
          dot += v * (a.scale * __ldg(dw + j));
        }
        sum = O::sum(sum);
        dot = O::sum(dot) / sum;
      }
      for (int j = l; j < a.topk; j += LPT) {
        if (!inside(j) || constant) continue;
        const float x = chosen(j), g = a.scale * __ldg(dw + j);
        float d = part(x) / sum * (a.renorm ? g - dot : g);
        if (!a.softmax) {
          const float e = expf(-fabsf(x));  // 1 - s
          d *= (x > 0.0f ? e : 1.0f) / (1.0f + e);
        }
        if (!sparse) out[ids[j]] = d;
        else if (here) a.dlogits[t * a.E + ids[j]] += d;
      }
    }
    if (sparse) continue;
    __syncwarp();
    if (here) {
      float* dst = a.dlogits + t * a.E;
      if (a.E % 4 == 0) {
        for (int e = l * 4; e < a.E; e += LPT * 4) {
          float4 v = *reinterpret_cast<const float4*>(out + e);
          if (a.accumulate) {
            const float4 o = *reinterpret_cast<const float4*>(dst + e);
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
          }
          *reinterpret_cast<float4*>(dst + e) = v;
        }
      } else {
        for (int e = l; e < a.E; e += LPT) dst[e] = a.accumulate ? dst[e] + out[e] : out[e];
      }
    }
    __syncwarp();
    if (!every)
      for (int j = l; j < a.topk; j += LPT)
        if (inside(j)) out[ids[j]] = 0.0f;
  }
}

flux_status_t check_gate(int T, int E, int topk, int score, float scale, const float* logits) {
  if (T < 0 || E < 1 || E > FLUX_MAX_EXPERTS || topk < 1 || topk > E) return FLUX_ERR_INVALID_ARG;
  if (score != FLUX_SCORE_SOFTMAX && score != FLUX_SCORE_SIGMOID) return FLUX_ERR_INVALID_ARG;
  if (!isfinite(scale)) return FLUX_ERR_INVALID_ARG;
  if (T > 0 && logits == nullptr) return FLUX_ERR_INVALID_ARG;
  return aligned16(logits) ? FLUX_OK : FLUX_ERR_UNSUPPORTED;
}

template <int LPT, int NC>
flux_status_t launch_gate(const GroupGateArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int TPC = GG_WARPS * (32 / LPT);
  constexpr auto kernel = group_gate_kernel<LPT, NC>;
  const size_t smem = TPC * gate_token_bytes(a.row, a.topk);
  static OncePerDevice once;
  const cudaError_t attr = once(dev.device, [&dev] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dev.max_smem_optin));
  });
  if (attr != cudaSuccess) return cuda_fail(attr);
  const int per_sm = static_cast<int>(std::max<size_t>(1, std::min<size_t>(NC <= 8 ? 5 : 2, (227u << 10) / (smem + 1024))));
  const int grid = std::min(ceil_div(a.T, TPC), GG_SMS * per_sm);
  const cudaError_t e = launch_behind(kernel, dim3(grid), GG_THREADS, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int LPT>
flux_status_t launch_gate_bwd(const GroupGateArgs& a, cudaStream_t s) {
  constexpr int TPC = GG_WARPS * (32 / LPT);
  const size_t smem = static_cast<size_t>(TPC) * ((a.E + 3) & ~3) * sizeof(float);  // at most 32 KB
  const int grid = std::min(ceil_div(a.T, TPC), GG_SMS * 4);
  const cudaError_t e = launch_behind(group_gate_bwd_kernel<LPT>, dim3(grid), GG_THREADS, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
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
  a.G = groups;
  a.kept = topk_groups;
  a.top = group_top;
  a.n = E / groups;
  a.div_n = ((1u << 20) + a.n - 1) / a.n;
  a.softmax = score == FLUX_SCORE_SOFTMAX;
  a.renorm = renorm != 0;
  a.scale = scale;
  const int lpt = E <= 64 ? 8 : 32;
  a.lpg = lpt;  // lanes of a group: as many as let all groups be ranked at once, at least one
  while (a.lpg > 1 && a.lpg * groups > lpt) a.lpg /= 2;
  a.pad = topk_groups < groups ? a.lpg : 0;
  a.row = E + groups * a.pad;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int each = ceil_div(topk_groups * a.n, lpt);  // candidates of a lane
  if (lpt == 8) {
    if (each <= 1) return launch_gate<8, 1>(a, dev, s);
    if (each <= 2) return launch_gate<8, 2>(a, dev, s);
    if (each <= 4) return launch_gate<8, 4>(a, dev, s);
    return launch_gate<8, 8>(a, dev, s);
  }
  if (each <= 4) return launch_gate<32, 4>(a, dev, s);
  if (each <= 8) return launch_gate<32, 8>(a, dev, s);
  if (each <= 16) return launch_gate<32, 16>(a, dev, s);
  return launch_gate<32, 32>(a, dev, s);
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
  return E <= 64 ? launch_gate_bwd<8>(a, s) : launch_gate_bwd<32>(a, s);
}
