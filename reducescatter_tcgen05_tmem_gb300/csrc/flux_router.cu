// The router's training side: balance and z losses with per-expert counts,
// and the gradient of the router scores.
//
// T tokens in S sequences of T / S, p = softmax of a token's E scores, m the
// token mask (1 or 0), n_s the kept tokens of sequence s, n all of them, c_se
// the kept slots of sequence s routed to expert e, P_se = sum_t m p_te / n_s:
//
//   balance = a E / (topk S) sum_s sum_e (c_se / n_s) P_se
//   z       = b / n sum_t m lse_t^2,          lse = log sum_e exp(score)
//
// The counts are constants of the gradient (they are piecewise constant in the
// scores), so with A_se = a E c_se / (topk S n_s^2)
//
//   d balance / d score_te = m p_te (A_se - sum_j p_tj A_sj)
//   d z / d score_te       = m p_te 2 b lse_t / n
//
// and the gate weights w = softmax over the chosen scores send their gradient
// dw to the chosen experts: w_j (dw_j - sum_i w_i dw_i).
//
// The rules for odd rows are the gate's: a NaN score counts as -inf; where the
// largest score is infinite the scores equal to it share p equally (all -inf:
// every expert).  Such a token has no z term and its scores get no gradient (p
// is constant around it).
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int RT_WARPS = 8, RT_THREADS = RT_WARPS * 32;
constexpr int RT_FWD_CTAS = 3 * 152, RT_BWD_CTAS = 5 * 152;  // at most this many: one wave
// the items of a lone sequence, and their sums, that its last CTA joins; more are
// joined by a second kernel
constexpr int RT_HERE_ITEMS = 64, RT_HERE_SUMS = 2048;
constexpr int JOIN_THREADS = 512, JOIN_FEW = 32;  // few items of a sequence: a thread adds all of an expert's
constexpr int JOIN_WIDE = 256, JOIN_NARROW = 32;  // experts of a joining block: few items, many

// A token's scores are held by LPT lanes, four by four: V vectors of four a
// lane.  Vectors of a row of 4 n experts are 16-byte loads of neighbours, other
// rows are read one score at a time, neighbours in neighbouring lanes.
template <int LPT, int V, bool VEC>
struct Lanes {
  static constexpr int TPW = 32 / LPT;             // tokens of a warp at a time
  static constexpr int TPC = RT_WARPS * TPW;       // of a CTA
  static constexpr int IDS = LPT <= 4 ? 2 : 1;     // expert ids that a lane loads ahead
  static __device__ __forceinline__ int expert(int l, int v, int i) {
    return VEC ? (v * LPT + l) * 4 + i : (v * 4 + i) * LPT + l;
  }
  // f[v][i] = row[expert], `other` past E
  static __device__ __forceinline__ void load(const float* row, int l, int E, float other, float (&f)[V][4]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (VEC) {
        const int e = expert(l, v, 0);
        const float4 q = e < E ? load_global(reinterpret_cast<const float4*>(row + e)) : make_float4(other, other, other, other);
        f[v][0] = q.x, f[v][1] = q.y, f[v][2] = q.z, f[v][3] = q.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[v][i] = expert(l, v, i) < E ? load_global(row + expert(l, v, i)) : other;
      }
    }
  }
  // sums over the LPT lanes of a token
  static __device__ __forceinline__ float sum(float x) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
  }
  static __device__ __forceinline__ float max(float x) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
  }
};

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// The hardware's 2^x and 1 / x (relative error about 2^-22; results below 2^-126
// are 0) and log2 x, whose error near x = 1 is about 2^-22 absolute: it is added to
// the largest score.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// How the forward pass cuts the tokens: `sub` items of `chunk` tokens per
// sequence, one CTA each.
struct BalancePlan {
  int sub, chunk, items, join_cols, cols;  // cols: blocks of join_cols experts of the joining kernel, 0 if there is none
  size_t probs, counts, kept, z, bal, seq_z, total;
};

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  float* loss;
  int32_t* counts;
  float* probs;
  int32_t* tokens;
  float* lse;
  uint32_t* hdr;
  // workspace: the items' sums, then one value per sequence (and column block)
  float* part_probs;
  int* part_counts;
  int* part_kept;
  float* part_z;
  float* part_bal;
  float* seq_z;
  uint32_t* arrived;  // header words: items of the one sequence, then sequences or blocks
  int E, topk, S, per, sub, chunk, cols;
  float balance_scale, z_coef;
};

// Arrival of this CTA, its stores made visible first, at a counter that
// `others` others arrive at too; true in the last one, which leaves the counter
// zero and sees the others' stores.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counter, int others, int* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const bool last = atomicAdd(counter, 1u) == static_cast<uint32_t>(others);
    if (last) *counter = 0u;
    *flag = last;
    __threadfence();
  }
  __syncthreads();
  return *flag != 0;
}

// Sums of two floats and an integer over the CTA, in a fixed order; in thread 0.
template <int THREADS>
__device__ __forceinline__ void cta_sums(float& x, float& y, int& n, float* smem) {
  x = warp_sum(x);
  y = warp_sum(y);
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    float* at = smem + (threadIdx.x >> 5) * 3;
    at[0] = x;
    at[1] = y;
    at[2] = __int_as_float(n);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < THREADS / 32; ++w) {
      x += smem[w * 3];
      y += smem[w * 3 + 1];
      n += __float_as_int(smem[w * 3 + 2]);
    }
  }
}

__device__ __forceinline__ void write_losses(const BalanceArgs& a, float bal, float z, int all) {
  a.loss[0] = bal * a.balance_scale;
  a.loss[1] = z * a.z_coef / static_cast<float>(max(all, 1));
  a.tokens[a.S] = all;
}

// The losses from the n parts of the balance loss and the sequences' z terms and
// counts, once all are there; leaves the parts zero.
template <int THREADS>
__device__ __forceinline__ void join_losses(const BalanceArgs& a, int n, float* smem) {
  float bal = 0.0f, z = 0.0f;
  int all = 0;
  for (int i = threadIdx.x; i < n; i += THREADS) {
    bal += __ldcg(a.part_bal + i);
    a.part_bal[i] = 0.0f;
  }
  for (int s = threadIdx.x; s < a.S; s += THREADS) {
    z += __ldcg(a.seq_z + s);
    a.seq_z[s] = 0.0f;
    all += __ldcg(a.tokens + s);
  }
  cta_sums<THREADS>(bal, z, all, smem);
  if (threadIdx.x == 0) write_losses(a, bal, z, all);
}

// Forward.  One read of the scores: a token's maximum, exponentials and their
// sum stay in the registers of its lanes, which add its probabilities to their
// own experts' sums.  An item's sums are joined over its warps in shared memory,
// a sequence's over its items by balance_join_kernel, or, where there is one
// sequence of few items, by the last of their CTAs; all in fixed orders.
//
// Bound by latency, with one group of tokens ahead in registers (issue slots 58 %,
// DRAM 65 %): 131072 x 256 in 64 masked sequences 30.6 us with the joining kernel, 4.6 TB/s
// (sums in double precision took 462); 4096 x 8 in one launch 5.9 us.
template <int LPT, int V, bool VEC>
__global__ void __launch_bounds__(RT_THREADS, V <= 4 ? 3 : 2)
balance_kernel(const __grid_constant__ BalanceArgs a) {
  using L = Lanes<LPT, V, VEC>;
  constexpr int WIDE = LPT * V * 4;  // experts the lanes have room for
  __shared__ float probs_w[RT_WARPS][WIDE];
  __shared__ int cnt[WIDE];
  __shared__ int kept_w[RT_WARPS];
  __shared__ float z_w[RT_WARPS];
  __shared__ float red[RT_WARPS * 3];
  __shared__ int flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPT, tg = lane / LPT;
  const int item = blockIdx.x, seq = item / a.sub, E = a.E;
  const int t0 = seq * a.per + (item - seq * a.sub) * a.chunk, t1 = t0 + min(a.chunk, (seq + 1) * a.per - t0);
  wait_for_previous();
  for (int e = threadIdx.x; e < WIDE; e += RT_THREADS) cnt[e] = 0;
  __syncthreads();
  float sums[V][4] = {};
  float z = 0.0f;
  int kept = 0;
  bool bad = false;
  // the next tokens' scores, mask and first expert are on their way while these
  // are at work
  float next[V][4];
  int next_id[L::IDS] = {}, next_mask = 1;
  auto fetch = [&](int t) {
    const size_t at = static_cast<size_t>(t < t1 ? t : t0);
    L::load(a.logits + at * E, l, E, -INFINITY, next);
#pragma unroll
    for (int k = 0; k < L::IDS; ++k)
      if (l + k * LPT < a.topk) next_id[k] = load_global(a.ids + at * a.topk + l + k * LPT);
    if (a.mask != nullptr) next_mask = load_global(a.mask + at);
  };
  if (t0 + warp * L::TPW < t1) fetch(t0 + warp * L::TPW + tg);
  for (int tw = t0 + warp * L::TPW; tw < t1; tw += L::TPC) {
    const int t = tw + tg;
    int id[L::IDS];
#pragma unroll
    for (int k = 0; k < L::IDS; ++k) id[k] = next_id[k];
    const bool here = t < t1, keep = here && next_mask != 0;
    float f[V][4];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[v][i] = fmaxf(next[v][i], -INFINITY);  // a NaN gives way to the other operand
        top = fmaxf(top, f[v][i]);
      }
    if (tw + L::TPC < t1) fetch(t + L::TPC);
    top = L::max(top);
    float s = 0.0f;
    if (!isinf(top)) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[v][i] = exp2_fast((f[v][i] - top) * LOG2E);
          s += f[v][i];
        }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[v][i] = L::expert(l, v, i) < E && f[v][i] == top ? 1.0f : 0.0f;
          s += f[v][i];
        }
    }
    s = L::sum(s);
    const float lse = isinf(top) ? top : top + log2_fast(s) * LN2;
    if (here && l == 0) a.lse[t] = lse;
    const float share = keep ? inverse_fast(s) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[v][i] += f[v][i] * share;
    if (keep) {
      if (l == 0) {
        ++kept;
        if (!isinf(top)) z += lse * lse;
      }
      auto count = [&](int e) {
        if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
        else bad = true;
      };
#pragma unroll
      for (int k = 0; k < L::IDS; ++k)
        if (l + k * LPT < a.topk) count(id[k]);
      for (int j = l + L::IDS * LPT; j < a.topk; j += LPT) count(load_global(a.ids + static_cast<size_t>(t) * a.topk + j));
    }
  }
  // tokens side by side in a warp, then the warps
#pragma unroll
  for (int o = LPT; o < 32; o <<= 1) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[v][i] += __shfl_xor_sync(0xFFFFFFFFu, sums[v][i], o);
  }
  z = warp_sum(z);
  kept = __reduce_add_sync(0xFFFFFFFFu, kept);
  if (lane < LPT) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) probs_w[warp][L::expert(l, v, i)] = sums[v][i];
  }
  if (lane == 0) {
    kept_w[warp] = kept;
    z_w[warp] = z;
  }
  if (bad) atomicCAS(a.hdr, 0u, static_cast<uint32_t>(FLUX_ERR_INVALID_ARG));
  __syncthreads();
  int n = 0;
  float z_item = 0.0f;
#pragma unroll
  for (int w = 0; w < RT_WARPS; ++w) {
    n += kept_w[w];
    z_item += z_w[w];
  }
  auto expert_sum = [&](int e) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < RT_WARPS; ++w) s += probs_w[w][e];
    return s;
  };
  float bal = 0.0f;
  auto write = [&](int e, float p, int c, int n_seq) {
    const float m = static_cast<float>(max(n_seq, 1));
    p /= m;
    a.probs[static_cast<size_t>(seq) * E + e] = p;
    a.counts[static_cast<size_t>(seq) * E + e] = c;
    bal += static_cast<float>(c) / m * p;
  };
  if (a.sub == 1) {
    for (int e = threadIdx.x; e < E; e += RT_THREADS) write(e, expert_sum(e), cnt[e], n);
  } else {
    for (int e = threadIdx.x; e < E; e += RT_THREADS) {
      a.part_probs[static_cast<size_t>(item) * E + e] = expert_sum(e);
      a.part_counts[static_cast<size_t>(item) * E + e] = cnt[e];
    }
    if (threadIdx.x == 0) {
      a.part_kept[item] = n;
      a.part_z[item] = z_item;
    }
    if (a.cols > 0) return;  // balance_join_kernel goes on
    if (!last_to_arrive(a.arrived, a.sub - 1, &flag)) return;
    const int i0 = seq * a.sub;
    if (warp == 0) {
      int n_seq = 0;
      float z_seq = 0.0f;
      for (int i = lane; i < a.sub; i += 32) {
        n_seq += __ldcg(a.part_kept + i0 + i);
        z_seq += __ldcg(a.part_z + i0 + i);
        a.part_kept[i0 + i] = 0;
        a.part_z[i0 + i] = 0.0f;
      }
      n_seq = __reduce_add_sync(0xFFFFFFFFu, n_seq);
      z_seq = warp_sum(z_seq);
      if (lane == 0) {
        kept_w[0] = n_seq;
        z_w[0] = z_seq;
      }
    }
    __syncthreads();
    n = kept_w[0];
    z_item = z_w[0];
    // an expert per warp, its items over the lanes, four experts in flight
    constexpr int BATCH = 4;
    for (int e0 = warp; e0 < E; e0 += RT_WARPS * BATCH) {
      float p[BATCH] = {};
      int c[BATCH] = {};
      for (int i = lane; i < a.sub; i += 32) {
        const size_t row = static_cast<size_t>(i0 + i) * E;
        float fp[BATCH];
        int fc[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int e = e0 + b * RT_WARPS;
          fp[b] = e < E ? __ldcg(a.part_probs + row + e) : 0.0f;
          fc[b] = e < E ? __ldcg(a.part_counts + row + e) : 0;
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int e = e0 + b * RT_WARPS;
          if (e < E) {
            a.part_probs[row + e] = 0.0f;
            a.part_counts[row + e] = 0;
          }
          p[b] += fp[b];
          c[b] += fc[b];
        }
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int e = e0 + b * RT_WARPS;
        p[b] = warp_sum(p[b]);
        c[b] = __reduce_add_sync(0xFFFFFFFFu, c[b]);
        if (lane == 0 && e < E) write(e, p[b], c[b], n);
      }
    }
  }
  float none = 0.0f;
  int no = 0;
  cta_sums<RT_THREADS>(bal, none, no, red);
  if (threadIdx.x == 0) {
    a.tokens[seq] = n;
    if (a.S == 1) {
      write_losses(a, bal, z_item, n);
    } else {
      a.part_bal[seq] = bal;
      a.seq_z[seq] = z_item;
    }
  }
  if (a.S == 1 || !last_to_arrive(a.arrived + 1, a.S - 1, &flag)) return;
  join_losses<RT_THREADS>(a, a.S, red);
}

// Joins the items' sums of COLS experts of one sequence, the items dealt out to
// JOIN_THREADS / COLS threads.  Latency: 3 us behind the forward kernel at 64
// sequences of 256 experts (8.6 us with cold caches).
template <int COLS>
__global__ void __launch_bounds__(JOIN_THREADS) balance_join_kernel(const __grid_constant__ BalanceArgs a) {
  constexpr int ROWS = JOIN_THREADS / COLS;
  __shared__ float probs_w[ROWS][COLS];
  __shared__ int cnt_w[ROWS][COLS];
  __shared__ float red[JOIN_THREADS / 32 * 3];
  __shared__ int kept, flag;
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
  const int seq = blockIdx.y, i0 = seq * a.sub, e = blockIdx.x * COLS + col;
  if (warp == 0) {  // every block of the sequence needs its count
    int n = 0;
    float z = 0.0f;
    for (int i = lane; i < a.sub; i += 32) {
      n += a.part_kept[i0 + i];
      z += a.part_z[i0 + i];
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    z = warp_sum(z);
    if (lane == 0) {
      kept = n;
      if (blockIdx.x == 0) {
        a.tokens[seq] = n;
        a.seq_z[seq] = z;
      }
    }
  }
  constexpr int BATCH = 8;
  float p = 0.0f;
  int c = 0;
  if (e < a.E) {
    for (int i1 = row; i1 < a.sub; i1 += ROWS * BATCH) {
      float fp[BATCH];
      int fc[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int i = i1 + b * ROWS;
        const size_t at = static_cast<size_t>(i0 + i) * a.E + e;
        fp[b] = i < a.sub ? a.part_probs[at] : 0.0f;
        fc[b] = i < a.sub ? a.part_counts[at] : 0;
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int i = i1 + b * ROWS;
        const size_t at = static_cast<size_t>(i0 + i) * a.E + e;
        if (i < a.sub) {
          a.part_probs[at] = 0.0f;
          a.part_counts[at] = 0;
        }
        p += fp[b];
        c += fc[b];
      }
    }
  }
  probs_w[row][col] = p;
  cnt_w[row][col] = c;
  __syncthreads();
  float bal = 0.0f, none = 0.0f;
  int no = 0;
  if (row == 0 && e < a.E) {
    for (int w = 1; w < ROWS; ++w) {
      p += probs_w[w][col];
      c += cnt_w[w][col];
    }
    const float n = static_cast<float>(max(kept, 1));
    p /= n;
    a.probs[static_cast<size_t>(seq) * a.E + e] = p;
    a.counts[static_cast<size_t>(seq) * a.E + e] = c;
    bal = static_cast<float>(c) / n * p;
  }
  cta_sums<JOIN_THREADS>(bal, none, no, red);
  if (threadIdx.x == 0) a.part_bal[seq * gridDim.x + blockIdx.x] = bal;
  if (!last_to_arrive(a.arrived + 1, gridDim.x * gridDim.y - 1, &flag)) return;
  for (int i = threadIdx.x; i < a.S * a.sub; i += JOIN_THREADS) {
    a.part_kept[i] = 0;
    a.part_z[i] = 0.0f;
  }
  join_losses<JOIN_THREADS>(a, gridDim.x * gridDim.y, red);
}

struct RouterBwdArgs {
  const float* logits;
  const int32_t* ids;
  const float* weights;
  const uint8_t* mask;
  const float* lse;
  const int32_t* counts;
  const int32_t* tokens;
  const float* dloss;
  const float* dweights;
  float* dlogits;
  int E, topk, S, per, sub, chunk;
  float balance_coef, z_coef;
};

// Backward: one read of the scores, one write of their gradient.  A CTA stays in
// one sequence, whose counts its lanes hold; the gate's terms of a token meet
// the others through a row of shared memory.  Bound by HBM: 131072 x 256 49 us,
// 5.8 TB/s.
template <int LPT, int V, bool VEC>
__global__ void __launch_bounds__(RT_THREADS, V <= 2 ? 5 : 2)
router_bwd_kernel(const __grid_constant__ RouterBwdArgs a) {
  using L = Lanes<LPT, V, VEC>;
  constexpr int WIDE = LPT * V * 4;
  __shared__ alignas(16) float gate[RT_WARPS * L::TPW][WIDE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPT, tg = lane / LPT;
  const int item = blockIdx.x, seq = item / a.sub, E = a.E;
  const int t0 = seq * a.per + (item - seq * a.sub) * a.chunk, t1 = t0 + min(a.chunk, (seq + 1) * a.per - t0);
  float* g = gate[warp * L::TPW + tg];
  wait_for_previous();
  const bool gates = a.dweights != nullptr;
  if (gates)
    for (int e = l; e < WIDE; e += LPT) g[e] = 0.0f;
  const float db = a.dloss != nullptr ? load_global(a.dloss) : 1.0f, dz = a.dloss != nullptr ? load_global(a.dloss + 1) : 1.0f;
  const float n = static_cast<float>(max(load_global(a.tokens + seq), 1)), all = static_cast<float>(max(load_global(a.tokens + a.S), 1));
  const float scale = db * (a.balance_coef * E / (static_cast<float>(a.topk) * a.S)) / (n * n);
  const float z_scale = dz * (2.0f * a.z_coef) / all;
  float A[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = L::expert(l, v, i);
      A[v][i] = e < E ? scale * static_cast<float>(load_global(a.counts + static_cast<size_t>(seq) * E + e)) : 0.0f;
    }
  __syncwarp();
  for (int tw = t0 + warp * L::TPW; tw < t1; tw += L::TPC) {
    const int t = tw + tg;
    const bool here = t < t1;
    const size_t row = static_cast<size_t>(here ? t : t0);
    const bool keep = here && (a.mask == nullptr || load_global(a.mask + t) != 0);
    const float lse = load_global(a.lse + row);
    const bool flat = isinf(lse) || lse != lse;
    float w = 0.0f, dw = 0.0f;
    int id = -1;
    if (gates && l < a.topk) {
      w = load_global(a.weights + row * a.topk + l);
      dw = load_global(a.dweights + row * a.topk + l);
      id = load_global(a.ids + row * a.topk + l);
    }
    float f[V][4];
    if (keep) {
      L::load(a.logits + row * E, l, E, -INFINITY, f);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) f[v][i] = -INFINITY;
    }
    float mean = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[v][i] = flat || f[v][i] != f[v][i] ? 0.0f : exp2_fast((f[v][i] - lse) * LOG2E);
        mean += f[v][i] * A[v][i];
      }
    mean = L::sum(mean);
    const float shift = (flat ? 0.0f : z_scale * lse) - mean;
    if (gates) {
      float dot = w * dw;
      for (int j = l + LPT; j < a.topk; j += LPT) dot += load_global(a.weights + row * a.topk + j) * load_global(a.dweights + row * a.topk + j);
      dot = L::sum(dot);
      if (here && !flat) {
        for (int j = l; j < a.topk; j += LPT) {
          if (j != l) {
            w = load_global(a.weights + row * a.topk + j);
            dw = load_global(a.dweights + row * a.topk + j);
            id = load_global(a.ids + row * a.topk + j);
          }
          if (id >= 0 && id < E) g[id] = w * (dw - dot);
        }
      }
      __syncwarp();
    }
    float* out = a.dlogits + row * E;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = f[v][i] * (A[v][i] + shift);
      if constexpr (VEC) {
        const int e = L::expert(l, v, 0);
        if (gates) {
          float4* at = reinterpret_cast<float4*>(g + e);
          const float4 q = *at;
          *at = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          d[0] += q.x, d[1] += q.y, d[2] += q.z, d[3] += q.w;
        }
        if (here && e < E) *reinterpret_cast<float4*>(out + e) = make_float4(d[0], d[1], d[2], d[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = L::expert(l, v, i);
          if (gates) {
            d[i] += g[e];
            g[e] = 0.0f;
          }
          if (here && e < E) out[e] = d[i];
        }
      }
    }
    if (gates) __syncwarp();
  }
}

template <int N>
using Int = std::integral_constant<int, N>;

// Calls f(LPT, V, VEC) for the lanes that hold a row of E scores.  Forward: four
// vectors a lane; what a token costs besides its scores (sums over its lanes,
// logarithm, inverse, counts) is shared by several tokens of the warp (131072 x
// 256: 31 us with two tokens a warp, 40 with one).  Backward has less of that
// and wants more lanes' loads on their way: one or two vectors (53 against 58 us).
template <bool FORWARD, typename F>
auto by_experts(int E, F&& f) {
  auto vec = [&](auto lpt, auto v) { return E % 4 == 0 ? f(lpt, v, std::true_type{}) : f(lpt, v, std::false_type{}); };
  if (E <= 4) return vec(Int<1>{}, Int<1>{});
  if constexpr (FORWARD) {
    if (E <= 8) return vec(Int<1>{}, Int<2>{});
    if (E <= 16) return vec(Int<1>{}, Int<4>{});
    if (E <= 32) return vec(Int<2>{}, Int<4>{});
    if (E <= 64) return vec(Int<4>{}, Int<4>{});
    if (E <= 128) return vec(Int<8>{}, Int<4>{});
    if (E <= 256) return vec(Int<16>{}, Int<4>{});
  } else {
    if (E <= 8) return vec(Int<2>{}, Int<1>{});
    if (E <= 16) return vec(Int<4>{}, Int<1>{});
    if (E <= 32) return vec(Int<8>{}, Int<1>{});
    if (E <= 64) return vec(Int<16>{}, Int<1>{});
    if (E <= 128) return vec(Int<32>{}, Int<1>{});
    if (E <= 256) return vec(Int<32>{}, Int<2>{});
  }
  if (E <= 512) return vec(Int<32>{}, Int<4>{});
  return vec(Int<32>{}, Int<8>{});
}

// Items of a sequence before its tokens are dealt out evenly: one wave of CTAs in
// all where S allows it, each with work for its warps.  Never fewer for more tokens.
template <bool FORWARD>
int most_items(int E, int per, int S) {
  const int tokens = by_experts<FORWARD>(E, [](auto lpt, auto, auto) { return RT_WARPS * 32 / decltype(lpt)::value; });
  return std::max(1, std::min((FORWARD ? RT_FWD_CTAS : RT_BWD_CTAS) / S, ceil_div(per, tokens)));
}

// Items of a sequence, equal but for the last.
template <bool FORWARD>
void cut_tokens(int E, int per, int S, int* sub, int* chunk) {
  *sub = most_items<FORWARD>(E, per, S);
  *chunk = ceil_div(per, *sub);
  *sub = ceil_div(per, *chunk);
}

BalancePlan balance_plan(int T, int E, int S) {
  BalancePlan p{};
  cut_tokens<true>(E, T / S, S, &p.sub, &p.chunk);
  p.items = p.sub * S;
  p.join_cols = p.sub <= JOIN_FEW ? JOIN_WIDE : JOIN_NARROW;
  const bool here = S == 1 && p.sub <= RT_HERE_ITEMS && static_cast<long long>(p.sub) * E <= RT_HERE_SUMS;
  p.cols = p.sub > 1 && !here ? (E + p.join_cols - 1) / p.join_cols : 0;
  size_t at = WS_HEADER;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, WS_ALIGN);
    return here;
  };
  // sizes by the items before they are made even, so that the workspace of a batch
  // is enough for every smaller one: 8664 tokens of 256 experts have 456 items, 9000 have 450
  const int most = most_items<true>(E, T / S, S);
  const size_t parts = most > 1 ? static_cast<size_t>(most) * S : 0;
  const int cols = most > 1 ? (E + JOIN_NARROW - 1) / JOIN_NARROW : 1;
  p.probs = take(sizeof(float) * parts * E);
  p.counts = take(sizeof(int) * parts * E);
  p.kept = take(sizeof(int) * parts);
  p.z = take(sizeof(float) * parts);
  p.bal = take(sizeof(float) * S * static_cast<size_t>(cols));
  p.seq_z = take(sizeof(float) * S);
  p.total = at;
  return p;
}

// the kernels count tokens in ints up to a CTA's group past the last one
constexpr int RT_MAX_TOKENS = INT_MAX - 2 * RT_THREADS + 1;

bool router_sizes_ok(int T, int E, int topk, int seqs) {
  return T >= 0 && T <= RT_MAX_TOKENS && E >= 1 && E <= FLUX_MAX_EXPERTS && topk >= 1 && topk <= E && seqs >= 1 && T % seqs == 0 &&
         static_cast<long long>(T) * topk < (1ll << 31);
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" size_t flux_moe_balance_workspace_size(int T, int E, int topk, int seqs) {
  if (!router_sizes_ok(T, E, topk, seqs)) return 0;
  return T == 0 ? WS_HEADER : balance_plan(T, E, seqs).total;
}

extern "C" flux_status_t flux_moe_balance_loss(int T, int E, int topk, int seqs, float balance_coef, float z_coef,
                                               const float* logits, const int32_t* topk_ids,
                                               const uint8_t* token_mask, float* loss, int32_t* counts, float* probs,
                                               int32_t* tokens, float* lse, void* workspace, size_t workspace_bytes,
                                               void* stream) {
  if (!router_sizes_ok(T, E, topk, seqs) || !isfinite(balance_coef) || !isfinite(z_coef)) return FLUX_ERR_INVALID_ARG;
  if (loss == nullptr || counts == nullptr || probs == nullptr || tokens == nullptr) return FLUX_ERR_INVALID_ARG;
  if (T > 0 && (logits == nullptr || topk_ids == nullptr || lse == nullptr)) return FLUX_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(token_mask) || !aligned16(loss) || !aligned16(counts) ||
      !aligned16(probs) || !aligned16(tokens) || !aligned16(lse))
    return FLUX_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (T == 0) {
    const size_t n = static_cast<size_t>(seqs) * E;
    if ((e = cudaMemsetAsync(loss, 0, 2 * sizeof(float), s)) != cudaSuccess ||
        (e = cudaMemsetAsync(counts, 0, n * sizeof(int32_t), s)) != cudaSuccess ||
        (e = cudaMemsetAsync(probs, 0, n * sizeof(float), s)) != cudaSuccess ||
        (e = cudaMemsetAsync(tokens, 0, (static_cast<size_t>(seqs) + 1) * sizeof(int32_t), s)) != cudaSuccess)
      return cuda_fail(e);
    return FLUX_OK;
  }
  const BalancePlan p = balance_plan(T, E, seqs);
  flux_status_t st = check_workspace(workspace, workspace_bytes, p.total);
  if (st != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  char* ws = static_cast<char*>(workspace);
  BalanceArgs a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.loss = loss;
  a.counts = counts;
  a.probs = probs;
  a.tokens = tokens;
  a.lse = lse;
  a.hdr = static_cast<uint32_t*>(workspace);
  a.part_probs = reinterpret_cast<float*>(ws + p.probs);
  a.part_counts = reinterpret_cast<int*>(ws + p.counts);
  a.part_kept = reinterpret_cast<int*>(ws + p.kept);
  a.part_z = reinterpret_cast<float*>(ws + p.z);
  a.part_bal = reinterpret_cast<float*>(ws + p.bal);
  a.seq_z = reinterpret_cast<float*>(ws + p.seq_z);
  a.arrived = static_cast<uint32_t*>(workspace) + WS_ARRIVED;
  a.E = E;
  a.topk = topk;
  a.S = seqs;
  a.per = T / seqs;
  a.sub = p.sub;
  a.chunk = p.chunk;
  a.cols = p.cols;
  a.balance_scale = static_cast<float>(static_cast<double>(balance_coef) * E / (static_cast<double>(topk) * seqs));
  a.z_coef = z_coef;
  by_experts<true>(E, [&](auto lpt, auto v, auto vec) {
    e = launch_behind(balance_kernel<decltype(lpt)::value, decltype(v)::value, decltype(vec)::value>, dim3(p.items), RT_THREADS, 0, s, a);
  });
  if (e != cudaSuccess) return cuda_fail(e);
  if (p.cols == 0) return FLUX_OK;
  e = launch_behind(p.join_cols == JOIN_WIDE ? balance_join_kernel<JOIN_WIDE> : balance_join_kernel<JOIN_NARROW>, dim3(p.cols, seqs), JOIN_THREADS, 0, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

extern "C" flux_status_t flux_moe_router_bwd(int T, int E, int topk, int seqs, float balance_coef, float z_coef,
                                             const float* logits, const int32_t* topk_ids, const float* topk_weights,
                                             const uint8_t* token_mask, const float* lse, const int32_t* counts,
                                             const int32_t* tokens, const float* dloss, const float* dweights,
                                             float* dlogits, void* stream) {
  if (!router_sizes_ok(T, E, topk, seqs) || !isfinite(balance_coef) || !isfinite(z_coef)) return FLUX_ERR_INVALID_ARG;
  if (T == 0) return FLUX_OK;
  if (logits == nullptr || lse == nullptr || counts == nullptr || tokens == nullptr || dlogits == nullptr)
    return FLUX_ERR_INVALID_ARG;
  if (dweights != nullptr && (topk_ids == nullptr || topk_weights == nullptr)) return FLUX_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(topk_weights) || !aligned16(token_mask) ||
      !aligned16(lse) || !aligned16(counts) || !aligned16(tokens) || !aligned16(dloss) || !aligned16(dweights) ||
      !aligned16(dlogits))
    return FLUX_ERR_UNSUPPORTED;
  DeviceInfo dev;
  flux_status_t st = current_device(&dev);
  if (st != FLUX_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouterBwdArgs a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.mask = token_mask;
  a.lse = lse;
  a.counts = counts;
  a.tokens = tokens;
  a.dloss = dloss;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.E = E;
  a.topk = topk;
  a.S = seqs;
  a.per = T / seqs;
  cut_tokens<false>(E, a.per, seqs, &a.sub, &a.chunk);
  a.balance_coef = balance_coef;
  a.z_coef = z_coef;
  cudaError_t e = cudaSuccess;
  by_experts<false>(E, [&](auto lpt, auto v, auto vec) {
    e = launch_behind(router_bwd_kernel<decltype(lpt)::value, decltype(v)::value, decltype(vec)::value>, dim3(a.sub * seqs), RT_THREADS, 0, s, a);
  });
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}
