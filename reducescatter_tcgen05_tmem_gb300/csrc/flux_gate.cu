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
// last one in and the first one out, are closer than the bounds it takes these two,
// or where there are more of them that token's whole choice, again in doubles.  Values
// made from equal scores and equal biases are equal in both, so that experts that tie cost
// nothing extra.  Groups whose ranks tie do: their two largest values in doubles, or where
// more than two are equal the whole choice (131072 x 256 of zero logits and biases 2.3 ms).
#include "flux_gate.cuh"

namespace flux {

namespace {

// One token of up to 64 experts to eight lanes, NC candidates each.  The lanes put the
// values into a row of shared memory, rank the groups from there, and take their
// candidates (those of the kept groups, in order) into registers for topk rounds of a
// maximum.  For long batches of what the octet form does not take: 131072 tokens, 4 of 48
// experts in 6 of 16 groups 85 us, a warp a token 108; 10 of 16 experts 31 and 55.
template <int NC>
__global__ void __launch_bounds__(GG_THREADS, 5)
group_gate_kernel(const __grid_constant__ GroupGateArgs a) {
  constexpr int LPT = 8, TPW = 32 / LPT;
  extern __shared__ uint4 smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPT, sub = lane / LPT;
  using O = Over<LPT>;
  const Rows r(reinterpret_cast<char*>(smem) + (warp * TPW + sub) * gate_token_bytes(a.row, a.topk), a.row, a.topk);
  const bool grouped = a.kept < a.G, biased = a.bias != nullptr, two = ranked_by_two(a, biased);
  const bool soft_row = a.softmax && (biased || !a.renorm || (grouped && two));
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
          r.val[at] = r.val[at] * inv + bias_of(a.bias, e);
        };
        if (a.E % 4 == 0) {
          for (int e = l * 4; e < a.E; e += LPT * 4) third(e), third(e + 1), third(e + 2), third(e + 3);
        } else {
          for (int e = l; e < a.E; e += LPT) third(e);
        }
      }
    } else {
      each_logit<LPT>(row, a.E, l, [&](int e, float x) {
        r.val[place(a, e)] = biased ? score(x) + bias_of(a.bias, e) : x;
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
        if (!two) m2 = 0.0f;
        else if (!biased) m1 = score(m1), m2 = score(m2);
        if (g < a.G && l % a.lpg == 0) {
          const float rank = fmaxf(m1 + m2, -INFINITY);
          const RankRange range(rank, m1, m2, unsure);
          r.rank[g] = rank;
          r.low[g] = range.low;
          r.high[g] = range.high;
        }
      }
      __syncwarp();
      uint32_t in = 0;
      float low = INFINITY, high = -INFINITY;
      for (int g = l; g < a.G; g += LPT) {
        const float mine = r.rank[g];
        int pos = 0;
        for (int o = 0; o < a.G; ++o) {
          const float other = r.rank[o];
          pos += other > mine || (other == mine && o < g);
        }
        if (pos < a.kept) {
          in |= 1u << g;
          low = fminf(low, r.low[g]);
        } else {
          high = fmaxf(high, r.high[g]);
        }
      }
      in = O::any(in);
      for (int g = l; g < a.G; g += LPT)
        if (in >> g & 1u) r.kept[__popc(in & ((1u << g) - 1u))] = g;
      low = -O::maxf(-low);
      high = O::maxf(high);
      __syncwarp();
      // (ranks that are logits are exact)
      if (biased || two) doubt = !ranks_apart(low, high);
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
      auto same = [&](int e, int f) { return load_global(row + e) == load_global(row + f) && bias_of(a.bias, e) == bias_of(a.bias, f); };
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
    if (doubt) choose64<LPT>(a, row, r.kept, r.pick, l, ((1u << LPT) - 1u) << (sub * LPT));
    __syncwarp();
    // the weights
    auto chosen = [&](int j) { return fmaxf(load_global(row + expert(j)), -INFINITY); };
    float peak = -INFINITY;
    if (a.renorm) {
      for (int j = l; j < a.topk; j += LPT) peak = fmaxf(peak, chosen(j));
      peak = O::maxf(peak);
    }
    auto weight = [&](float x) {
      if (a.renorm && (a.softmax ? isinf(peak) : peak == -INFINITY)) return x == peak ? 1.0f : 0.0f;
      if (a.softmax) return a.renorm ? expf(x - peak) : isinf(top) ? soft(x) : expf(x - top);
      return sigmoid_share(x, a.renorm ? peak : 0.0f);
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

// Words of a lane in shared memory, octet form: its logits, then its sorted lists of
// four (values, a NaN, their order; 8-byte stores).  No two of the eight lanes that read
// 16 bytes at a time meet in a bank.
template <int P>
__host__ __device__ constexpr int octet_pitch() {
  return P == 32 ? 52 : P == 16 ? 28 : 12;
}
__host__ __device__ inline int octet_words(int pitch) { return 32 * pitch + 4 * 8 + 8 + 32; }

// A group's rank in doubles, from its values from `least` on (x), of which there are y;
// the lanes of the group, lpg, have `mine` logits and biases each.  (Not inline: few
// tokens come here, and the others need not step over it.)
template <bool SOFT>
__device__ __noinline__ double2 group_rank64(const float* logit, const float* bias, int mine, float least, int lpg, float top, float inv, double sum) {
  int count = 0, e = 0, f = 0;
  for (int k = 0; k < mine; ++k) {
    const float x = fmaxf(logit[k], -INFINITY);
    const float c = (SOFT ? ex2((x - top) * G_LOG2E) * inv : rcp(1.0f + ex2(-x * G_LOG2E))) + bias[k];
    if (c < least) continue;
    ++count;
    f = e;
    e = k;
  }
  const double2 d = biased_scores64<SOFT>(logit[e], bias[e], logit[f], bias[f], top, sum);
  double exact = (count > 0 ? d.x : 0.0) + (count > 1 ? d.y : 0.0);
  for (int o = lpg >> 1; o > 0; o >>= 1) {
    count += __shfl_xor_sync(0xFFFFFFFFu, count, o);
    exact += __shfl_xor_sync(0xFFFFFFFFu, exact, o);
  }
  return make_double2(exact, count);
}

// Four tokens to a warp: a token's scores lie in neighbouring order in eight lanes, P
// at most in each, so that a group is one lane (or 2, 4 or 8) and most of the work is
// in the lanes' own registers.  Lists and rounds as in group_gate_wide_kernel.
// 131072 x 256 (8 of 256 in 4 of 8 groups) 83 us, of which the logits' bytes need 20:
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
  const bool grouped = a.kept < a.G, two = ranked_by_two(a, BIASED);
  const bool soft_row = SOFT && (BIASED || !a.renorm || (grouped && two));
  const int mine = min(a.per, max(a.E - l * a.per, 0));  // scores of this lane
  const bool full = a.per == P && a.E == 8 * P;
  const int group = l >> a.log_lpg, lpg = 1 << a.log_lpg;
  wait_for_previous();
  if constexpr (BIASED) {
    for (int i = threadIdx.x; i < 8 * (P + 4); i += GG_THREADS) {
      const int b = i / (P + 4), k = i - b * (P + 4), e = b * a.per + k;
      bias[i] = k < a.per && e < a.E ? bias_of(a.bias, e) : -INFINITY;
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
        const RankRange range(rank, m1, m2, unsure);
        const float low = -O::maxf(in ? -range.low : -INFINITY), high = O::maxf(in ? -INFINITY : range.high);
        doubt = !ranks_apart(low, high);
        // Groups next to the border: as in group_gate_wide_kernel.
        const bool here = doubt && !(SOFT && isinf(top));
        if (__any_sync(0xFFFFFFFFu, here)) {
          const double sum = SOFT ? softmax_total64<8>(row, a.E, l, top) : 0.0;
          const bool near = here && (in ? range.low <= high : range.high >= low);
          bool told = near;
          double exact;
          if constexpr (BIASED) {
            const int need = two ? 2 : 1;
            const double2 d = group_rank64<SOFT>(own, bias + l * (P + 4), near ? mine : 0, (two ? m2 : m1) - 2.0f * range.error, lpg, top, inv, sum);
            told = near && d.y == need;
            exact = d.x;
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
    float best = NAN;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= a.topk) break;
      best = head();
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
    // (as many taken as rounds, and none left for the last one: several in one round, where
    // every candidate is chosen)
    if (__any_sync(0xFFFFFFFFu, taken != a.topk || best != best)) {
      // several lists had the largest: the rounds again, the first expert takes it
      __syncwarp();
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        at[q] = lane * S + q * 6;
        h[q] = in ? own[q * 6] : NAN;
      }
      for (int j = 0; j < a.topk; ++j) {
        best = head();
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
        return load_global(row + f) == load_global(row + g) && bias_of(a.bias, f) == bias_of(a.bias, g);
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
      w = peak == -INFINITY ? 1.0f : sigmoid_share(x, peak);
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
      const float up = a.scale * load_global(a.dweights + t * a.topk + l);
      if (id >= 0) {  // (what lies beside another id may be anything)
        g = up;
        x = fmaxf(load_global(a.logits + t * a.E + id), -INFINITY);
      }
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
      // (what lies beside an id outside the experts may be anything)
      return e >= 0 && e < a.E ? Slot{e, g, fmaxf(load_global(row + e), -INFINITY)} : Slot{-1, 0.0f, -INFINITY};
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
  return group_gate_wide(a, dev, s);
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
