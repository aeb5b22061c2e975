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
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int RT_WARPS = 8, RT_THREADS = RT_WARPS * 32;
constexpr int RT_ITEMS = 608;  // about this many partial sums of the forward pass

// How the forward pass cuts the tokens: `sub` items of `chunk` tokens per sequence.
struct BalancePlan {
  int sub, chunk, items;
  size_t probs, counts, kept, z, total;
};

BalancePlan balance_plan(int T, int E, int S) {
  BalancePlan p{};
  const int per = T / S;
  p.sub = std::max(1, std::min((RT_ITEMS + S - 1) / S, (per + RT_WARPS - 1) / RT_WARPS));
  p.chunk = std::max(1, (per + p.sub - 1) / p.sub);
  p.sub = std::max(1, (per + p.chunk - 1) / p.chunk);
  p.items = p.sub * S;
  size_t at = WS_HEADER;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, WS_ALIGN);
    return here;
  };
  p.probs = take(sizeof(float) * p.items * static_cast<size_t>(E));
  p.counts = take(sizeof(int) * p.items * static_cast<size_t>(E));
  p.kept = take(sizeof(int) * p.items);
  p.z = take(sizeof(float) * p.items);
  p.total = at;
  return p;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// One item per CTA, one token per warp at a time; lane i holds the experts
// i, i + 32, ... and the sums of their probabilities.
template <int N>
__global__ void __launch_bounds__(RT_THREADS)
balance_kernel(int T, int E, int topk, int per, int sub, int chunk, const float* __restrict__ logits,
               const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, float* __restrict__ lse,
               float* part_probs, int* part_counts, int* part_kept, float* part_z, uint32_t* hdr) {
  extern __shared__ float sm[];  // E counts, then RT_WARPS x E probability sums
  int* cnt = reinterpret_cast<int*>(sm);
  float* probs = sm + E;
  __shared__ int kept_w[RT_WARPS];
  __shared__ float z_w[RT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = blockIdx.x, seq = item / sub;
  const int t0 = seq * per + (item - seq * sub) * chunk, t1 = min(t0 + chunk, (seq + 1) * per);
  for (int e = threadIdx.x; e < E; e += RT_THREADS) cnt[e] = 0;
  __syncthreads();
  float sum[N] = {};
  float z = 0.0f;
  int kept = 0;
  bool bad = false;
  for (int t = t0 + warp; t < t1; t += RT_WARPS) {
    const float* row = logits + static_cast<size_t>(t) * E;
    float v[N];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
      if (v[i] != v[i]) v[i] = -INFINITY;
      top = fmaxf(top, v[i]);
    }
    top = warp_max(top);
    const bool inf_top = isinf(top);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      v[i] = e >= E ? 0.0f : inf_top ? (v[i] == top ? 1.0f : 0.0f) : expf(v[i] - top);
      s += v[i];
    }
    s = warp_sum(s);
    const float l = inf_top ? top : top + logf(s);
    if (lane == 0) lse[t] = l;
    if (mask == nullptr || mask[t] != 0) {
      const float inv = 1.0f / s;
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] += v[i] * inv;
      ++kept;
      if (!inf_top) z += l * l;
      for (int j = lane; j < topk; j += 32) {
        const int e = ids[static_cast<size_t>(t) * topk + j];
        if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
        else bad = true;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    if (e < E) probs[warp * E + e] = sum[i];
  }
  if (lane == 0) {
    kept_w[warp] = kept;
    z_w[warp] = z;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += RT_THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < RT_WARPS; ++w) s += probs[w * E + e];
    part_probs[static_cast<size_t>(item) * E + e] = s;
    part_counts[static_cast<size_t>(item) * E + e] = cnt[e];
  }
  if (threadIdx.x == 0) {
    int k = 0;
    float s = 0.0f;
    for (int w = 0; w < RT_WARPS; ++w) {
      k += kept_w[w];
      s += z_w[w];
    }
    part_kept[item] = k;
    part_z[item] = s;
  }
  if (bad) atomicCAS(hdr, 0u, static_cast<uint32_t>(FLUX_ERR_INVALID_ARG));
}

// One CTA joins the items of each sequence in order, then the sequences, and
// leaves the partial sums zero.
__global__ void __launch_bounds__(1024)
balance_sums_kernel(int E, int topk, int S, int sub, float balance_coef, float z_coef, float* part_probs,
                    int* part_counts, int* part_kept, float* part_z, float* loss, int32_t* counts, float* probs,
                    int32_t* tokens) {
  __shared__ double warp_part[32];
  __shared__ int kept;
  double bal = 0.0;  // thread 0 .. E - 1: their expert's terms
  int all = 0;
  double z = 0.0;
  for (int s = 0; s < S; ++s) {
    if (threadIdx.x == 0) {
      int k = 0;
      for (int i = s * sub; i < (s + 1) * sub; ++i) {
        k += part_kept[i];
        z += part_z[i];
        part_kept[i] = 0;
        part_z[i] = 0.0f;
      }
      kept = k;
      all += k;
      tokens[s] = k;
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e < E) {
      float p = 0.0f;
      int c = 0;
      for (int i = s * sub; i < (s + 1) * sub; ++i) {
        const size_t at = static_cast<size_t>(i) * E + e;
        p += part_probs[at];
        c += part_counts[at];
        part_probs[at] = 0.0f;
        part_counts[at] = 0;
      }
      const float n = static_cast<float>(max(kept, 1));
      p /= n;
      probs[static_cast<size_t>(s) * E + e] = p;
      counts[static_cast<size_t>(s) * E + e] = c;
      bal += static_cast<double>(c) / n * p;
    }
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bal += __shfl_xor_sync(0xFFFFFFFFu, bal, o);
  if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x >> 5] = bal;
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0;
    for (int w = 0; w < 32; ++w) b += warp_part[w];
    loss[0] = static_cast<float>(b * balance_coef * E / (static_cast<double>(topk) * S));
    loss[1] = static_cast<float>(z * z_coef / max(all, 1));
    tokens[S] = all;
  }
}

// One token per warp: the loss terms first, then the gate's.
template <int N>
__global__ void __launch_bounds__(RT_THREADS)
router_bwd_kernel(int T, int E, int topk, int S, int per, float balance_coef, float z_coef,
                  const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ weights,
                  const uint8_t* __restrict__ mask, const float* __restrict__ lse, const int32_t* __restrict__ counts,
                  const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                  const float* __restrict__ dweights, float* __restrict__ dlogits) {
  extern __shared__ float sm[];  // RT_WARPS x E: the gate's terms of the warp's token
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* gate = sm + warp * E;
  const float db = dloss != nullptr ? dloss[0] : 1.0f, dz = dloss != nullptr ? dloss[1] : 1.0f;
  const float nall = static_cast<float>(max(tokens[S], 1));
  if (dweights != nullptr) {
    for (int e = lane; e < E; e += 32) gate[e] = 0.0f;
    __syncwarp();
  }
  for (long long t = static_cast<long long>(blockIdx.x) * RT_WARPS + warp; t < T;
       t += static_cast<long long>(gridDim.x) * RT_WARPS) {
    const int seq = static_cast<int>(t) / per;
    const float* row = logits + static_cast<size_t>(t) * E;
    const float l = lse[t];
    const bool flat = isinf(l) || l != l;
    const bool keep = !flat && (mask == nullptr || mask[t] != 0);
    float p[N], a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = a[i] = 0.0f;
    float mean = 0.0f, zt = 0.0f;
    if (keep) {
      const float n = static_cast<float>(max(tokens[seq], 1));
      const float scale = db * (balance_coef * E / (static_cast<float>(topk) * S)) / (n * n);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        if (e < E) {
          const float v = __ldg(row + e);
          p[i] = v != v ? 0.0f : expf(v - l);
          a[i] = scale * static_cast<float>(counts[static_cast<size_t>(seq) * E + e]);
          mean += p[i] * a[i];
        }
      }
      mean = warp_sum(mean);
      zt = dz * (2.0f * z_coef) * l / nall;
    }
    if (dweights != nullptr && !flat) {
      const float* w = weights + static_cast<size_t>(t) * topk;
      const float* dw = dweights + static_cast<size_t>(t) * topk;
      const int32_t* id = ids + static_cast<size_t>(t) * topk;
      float dot = 0.0f;
      for (int j = lane; j < topk; j += 32) dot += w[j] * dw[j];
      dot = warp_sum(dot);
      for (int j = lane; j < topk; j += 32) {
        const int e = id[j];
        if (e >= 0 && e < E) gate[e] = w[j] * (dw[j] - dot);
      }
      __syncwarp();
    }
    float* out = dlogits + static_cast<size_t>(t) * E;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      if (e < E) {
        float d = p[i] * (a[i] - mean + zt);
        if (dweights != nullptr) {
          d += gate[e];
          gate[e] = 0.0f;
        }
        out[e] = d;
      }
    }
    __syncwarp();
  }
}

template <typename F>
flux_status_t by_experts(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

bool router_sizes_ok(int T, int E, int topk, int seqs) {
  return T >= 0 && E >= 1 && E <= FLUX_MAX_EXPERTS && topk >= 1 && topk <= E && seqs >= 1 && T % seqs == 0 &&
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
        (e = cudaMemsetAsync(tokens, 0, (seqs + 1) * sizeof(int32_t), s)) != cudaSuccess)
      return cuda_fail(e);
    return FLUX_OK;
  }
  const BalancePlan p = balance_plan(T, E, seqs);
  flux_status_t st = check_workspace(workspace, workspace_bytes, p.total);
  if (st != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  char* ws = static_cast<char*>(workspace);
  float* part_probs = reinterpret_cast<float*>(ws + p.probs);
  int* part_counts = reinterpret_cast<int*>(ws + p.counts);
  int* part_kept = reinterpret_cast<int*>(ws + p.kept);
  float* part_z = reinterpret_cast<float*>(ws + p.z);
  st = by_experts(E, [&](auto n) {
    const size_t smem = sizeof(float) * E * (1 + RT_WARPS);
    balance_kernel<decltype(n)::value><<<p.items, RT_THREADS, smem, s>>>(
        T, E, topk, T / seqs, p.sub, p.chunk, logits, topk_ids, token_mask, lse, part_probs, part_counts, part_kept,
        part_z, static_cast<uint32_t*>(workspace));
    const cudaError_t le = cudaGetLastError();
    return le == cudaSuccess ? FLUX_OK : cuda_fail(le);
  });
  if (st != FLUX_OK) return st;
  balance_sums_kernel<<<1, 1024, 0, s>>>(E, topk, seqs, p.sub, balance_coef, z_coef, part_probs, part_counts,
                                         part_kept, part_z, loss, counts, probs, tokens);
  e = cudaGetLastError();
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
  return by_experts(E, [&](auto n) {
    const int grid = std::min((T + RT_WARPS - 1) / RT_WARPS, dev.sm_count * 8);
    router_bwd_kernel<decltype(n)::value><<<grid, RT_THREADS, sizeof(float) * E * RT_WARPS, s>>>(
        T, E, topk, seqs, T / seqs, balance_coef, z_coef, logits, topk_ids, topk_weights, token_mask, lse, counts,
        tokens, dloss, dweights, dlogits);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  });
}
