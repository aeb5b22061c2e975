// Routing with expert groups, a warp a token (flux_gate.cu has the formulas and says
// which calls come here).
#include "flux_gate.cuh"

namespace flux {

namespace {

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
  const bool two = ranked_by_two(a, BIASED);
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
      bias[p] = p < places && p - group_of(p) * a.np < a.n ? bias_of(a.bias, id_of(p)) : -INFINITY;
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
        const RankRange range(rank, m1, m2, unsure);
        const float low = -warp_largest(in ? -range.low : NAN), high = warp_largest(in || g >= a.G ? NAN : range.high);
        doubt = !ranks_apart(low, high);
        // Groups next to the border: their ranks in doubles, from their two largest values
        // (unless a third is next to the second) or their largest, wherever they lie.
        if (doubt && !(SOFT && isinf(top))) {
          const double sum = SOFT ? softmax_total64<32>(a.logits + static_cast<size_t>(t) * a.E, a.E, lane, top) : 0.0;
          const bool near = g < a.G && (in ? range.low <= high : range.high >= low);
          bool told = near;
          double exact;
          if constexpr (BIASED) {
            const float least = (two ? m2 : m1) - 2.0f * range.error;
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
    // taken than rounds tell, or (where every candidate is chosen) a last round that found
    // none, and the rounds are gone through again with care.
    float best = NAN;
    for (int j0 = 0; j0 < a.topk; j0 += 8) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (j0 + u >= a.topk) break;
        best = warp_largest(head());
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
    if (__reduce_add_sync(0xFFFFFFFFu, taken) != a.topk || best != best) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        at[q] = (q * 32 + lane) * 5;
        h[q] = list[at[q]];
      }
      for (int j = 0; j < a.topk; ++j) {
        best = warp_largest(head());
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
    // The weights, with the rules of group_gate_kernel.
    auto logit = [&](int e) { return fmaxf(raw[e], -INFINITY); };
    float peak = 0.0f;
    auto weight = [&](float x) {
      if constexpr (SOFT) {
        if (a.renorm) return isinf(peak) ? (x == peak ? 1.0f : 0.0f) : expf(x - peak);
        return isinf(top) ? (x == top ? 1.0f : 0.0f) : expf(x - top);
      } else {
        return peak == -INFINITY ? 1.0f : sigmoid_share(x, peak);
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
  return launch_wide<0, GROUPED ? 9 : 8, GROUPED>(a, dev, s);  // (groups may have more than 1024 places)
}

}  // namespace

flux_status_t group_gate_wide(GroupGateArgs a, const DeviceInfo& dev, cudaStream_t s) {
  const bool grouped = a.kept < a.G;
  a.np = (a.n + 3) / 4 * 4;
  a.div_np = ((1u << 20) + a.np - 1) / a.np;
  a.pad = !grouped || a.lpg >= 8 ? 0 : (4 * a.lpg - a.np % 32 + 32) % 32;
  a.vecs = ceil_div(a.G * a.np, 128);
  a.trips = ceil_div(a.np, 4 * a.lpg);
  a.rivals = ceil_div(a.G, a.lpg);
  a.row = !grouped ? 0 : 128 * a.vecs + (128 * a.vecs - 4) / a.np * a.pad;  // values of every place
  return grouped ? launch_wide<true>(a, dev, s) : launch_wide<false>(a, dev, s);
}

}  // namespace flux
