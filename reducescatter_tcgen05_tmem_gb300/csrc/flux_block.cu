// Norms around a block: the block's output is normalised, gated and added to
// the scaled residual stream, and the sum is normalised for the next block.
//
//   z  = y r_y w_post          r_y = (mean y^2 + eps)^-1/2   (z = y without post-norm)
//   x' = rho x + g z
//   u  = x' r_x w_pre          r_x = (mean x'^2 + eps)^-1/2
//
// and, with d = dx' + r_x (w_pre du - xn mean(w_pre du xn)), xn = x' r_x,
// yn = y r_y, the gradients
//
//   dx = rho d                 dy = r_y (c - yn mean(c yn)),  c = d g w_post
//   dw_pre = sum_t du xn       dw_post = sum_t d g yn
//   dg = sum_t d z             drho = sum_t,h d x
//
// Every element takes part in two (forward) or two dependent (backward) sums
// over its row, so a row is held by one team of warps from its load to its
// store and crosses HBM once in each direction.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

constexpr int BLOCK_MAX_H = FLUX_BLOCK_MAX_H;
constexpr int BN_MAX_CTAS = 304;  // persistent backward grid: at most two CTAs on each of 152 SMs

struct BlockNormArgs {
  const void* x[FLUX_MAX_RANKS];
  const void* y[FLUX_MAX_RANKS];
  void* out_a[FLUX_MAX_RANKS];  // forward: x';   backward: dx
  void* out_b[FLUX_MAX_RANKS];  // forward: u;    backward: dy
  const void* dx_out[FLUX_MAX_RANKS];
  const void* du[FLUX_MAX_RANKS];
  const void* w_post;
  const void* gate;
  const float* res_scale;
  const void* w_pre;
  float* rstd_y;
  float* rstd_x;
  float *dw_post, *dgate, *dres, *dw_pre;
  // backward partial sums (workspace)
  float *part_pre, *part_post, *part_gate;
  double *part_res, *part_scalar;
  int T, H, rows_per_rank;
  int post_norm, has_y, has_u, has_dx_out;
  int gate_per, gate_cols;  // rows of one gate row; 1 or H
  int items, sub, chunk, item_rows;  // items of `chunk` rows, `sub` in each run of `item_rows` rows
  float eps;
};

namespace {

// A row is held by a team of W warps; a CTA has one to eight teams.
template <int W>
struct Team {
  static constexpr int THREADS = W * 32;
  static constexpr int CTA = W <= 8 ? 256 : W * 32;
  static constexpr int COUNT = CTA / THREADS;
};

template <int DT>
__device__ __forceinline__ void load8(const void* base, size_t elem, float (&f)[8]) {
  unpack8<DT>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem)), f);
}

// Weights of the vector at column `col`, or ones.
template <int DT>
__device__ __forceinline__ void load_or_one(const void* base, size_t elem, float (&f)[8]) {
  if (base != nullptr) {
    load8<DT>(base, elem, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  }
}

// Gate of row t at column `col`.
template <int DT>
__device__ __forceinline__ void load_gate(const BlockNormArgs& a, int t, int col, float (&f)[8]) {
  if (a.gate == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  } else if (a.gate_cols == 1) {
    const float g = load16<DT>(a.gate, t / a.gate_per);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = g;
  } else {
    load8<DT>(a.gate, static_cast<size_t>(t / a.gate_per) * a.H + col, f);
  }
}

// Forward: one team of W warps per row, V vectors of 8 columns per thread.
template <int DT, int W, int V>
__global__ void __launch_bounds__(Team<W>::CTA)
block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  __shared__ float red[Team<W>::COUNT][2 * W];
  const int team = threadIdx.x / Team<W>::THREADS, lane = threadIdx.x % Team<W>::THREADS;
  const int wit = lane / 32;
  int turn = 0;
  const float rho = a.res_scale != nullptr ? __ldg(a.res_scale) : 1.0f;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  for (long long t = static_cast<long long>(blockIdx.x) * Team<W>::COUNT + team; t < a.T;
       t += static_cast<long long>(gridDim.x) * Team<W>::COUNT) {
    const int rank = static_cast<int>(t) / a.rows_per_rank;
    const size_t row = static_cast<size_t>(static_cast<int>(t) - rank * a.rows_per_rank) * a.H;
    float x1[V][8];
    float ry = 1.0f;
    if (a.has_y) {
      float ys[V][8];
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * Team<W>::THREADS + lane) * 8;
        if (col < a.H) {
          load8<DT>(a.y[rank], row + col, ys[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += ys[v][i] * ys[v][i];
        }
      }
      if (a.post_norm) {
        team_sum<W>(s, red[team], turn, team, wit);
        ry = rsqrtf(s[0] * inv_h + a.eps);
        if (lane == 0 && a.rstd_y != nullptr) a.rstd_y[t] = ry;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * Team<W>::THREADS + lane) * 8;
        if (col < a.H) {
          float w[8], g[8];
          load8<DT>(a.x[rank], row + col, x1[v]);
          load_or_one<DT>(a.w_post, col, w);
          load_gate<DT>(a, static_cast<int>(t), col, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) x1[v][i] = rho * x1[v][i] + g[i] * (ys[v][i] * ry * w[i]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_a[rank]) + row + col) = pack8<DT>(x1[v]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * Team<W>::THREADS + lane) * 8;
        if (col < a.H) load8<DT>(a.x[rank], row + col, x1[v]);
      }
    }
    if (!a.has_u) continue;
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * Team<W>::THREADS + lane) * 8;
      if (col < a.H) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += x1[v][i] * x1[v][i];
      }
    }
    team_sum<W>(s, red[team], turn, team, wit);
    const float rx = rsqrtf(s[0] * inv_h + a.eps);
    if (lane == 0 && a.rstd_x != nullptr) a.rstd_x[t] = rx;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * Team<W>::THREADS + lane) * 8;
      if (col < a.H) {
        float w[8];
        load_or_one<DT>(a.w_pre, col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = x1[v][i] * rx * w[i];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_b[rank]) + row + col) = pack8<DT>(w);
      }
    }
  }
}

// Backward.  A CTA walks items of `chunk` consecutive rows that share a gate
// row; its teams take the item's rows in turn, and every thread keeps the sums
// of its own columns in registers:
//   pre  = sum du xn of all its rows (dw_pre);
//   post = sum d yn: with one gate row for all tokens, dw_post = g post and
//          dg = w_post post, so one sum serves both; with a gate per row it is
//          sum d g yn;
//   A    = MULTI (a CTA can meet several rows of a gate per column): sum d yn
//          of the current item, from which dg = w_post A and post += g A.
// The teams' sums are joined in shared memory and the CTAs' by
// block_norm_sums_kernel, both in a fixed order, so repeat calls give the same
// bits.
template <int DT, int W, int V, bool MULTI>
__global__ void __launch_bounds__(Team<W>::CTA)
block_norm_bwd_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int TT = Team<W>::THREADS, TEAMS = Team<W>::COUNT;
  __shared__ float red1[TEAMS][2 * W], red3[TEAMS][6 * W];
  __shared__ double sums[TEAMS];
  __shared__ float join[TEAMS > 1 ? TEAMS * TT * V * 8 : 1];
  const int team = threadIdx.x / TT, lane = threadIdx.x % TT, wit = lane / 32;
  int turn1 = 0, turn3 = 0;
  const float rho = a.res_scale != nullptr ? __ldg(a.res_scale) : 1.0f;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool row_gate = a.gate != nullptr && a.gate_cols == 1;
  const bool item_scalar = row_gate && a.gate_per > 1;
  float pre[V][8] = {}, post[V][8] = {};
  double res = 0.0;

  // dst[col] = (w ? w[col] : 1) * sum over teams of acc
  auto join_teams = [&](const float (&acc)[V][8], float* dst, const void* w) {
    if constexpr (TEAMS > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * TT + lane) * 8;
        if (col < a.H) {
#pragma unroll
          for (int i = 0; i < 8; ++i) join[team * a.H + col + i] = acc[v][i];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += Team<W>::CTA) {
        float s = join[c];
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) s += join[k * a.H + c];
        dst[c] = w != nullptr ? s * load16<DT>(w, c) : s;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * TT + lane) * 8;
        if (col < a.H) {
          float f[8];
          load_or_one<DT>(w, col, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= acc[v][i];
          reinterpret_cast<float4*>(dst + col)[0] = make_float4(f[0], f[1], f[2], f[3]);
          reinterpret_cast<float4*>(dst + col)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    }
  };
  auto join_scalar = [&](double v, double* dst) {
    if (lane == 0) sums[team] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = sums[0];
      for (int k = 1; k < TEAMS; ++k) s += sums[k];
      *dst = s;
    }
    __syncthreads();
  };

  for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int run = item / a.sub;
    const int t0 = run * a.item_rows + (item - run * a.sub) * a.chunk;
    const int t1 = min(t0 + a.chunk, (run + 1) * a.item_rows);
    float A[MULTI ? V : 1][8] = {};
    double scalar = 0.0;
    for (int t = t0 + team; t < t1; t += TEAMS) {
      const int rank = t / a.rows_per_rank;
      const size_t row = static_cast<size_t>(t - rank * a.rows_per_rank) * a.H;
      const float ry = a.post_norm ? __ldg(a.rstd_y + t) : 1.0f;
      const float rx = a.has_u ? __ldg(a.rstd_x + t) : 0.0f;
      float m1 = 0.0f;
      if (a.has_u) {
        float s1[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int col = (v * TT + lane) * 8;
          if (col < a.H) {
            float x[8], y[8], du[8], g[8], w[8], wp[8];
            load8<DT>(a.x[rank], row + col, x);
            load8<DT>(a.du[rank], row + col, du);
            load_or_one<DT>(a.w_pre, col, wp);
            if (a.has_y) {
              load8<DT>(a.y[rank], row + col, y);
              load_or_one<DT>(a.w_post, col, w);
              load_gate<DT>(a, t, col, g);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x1 = a.has_y ? rho * x[i] + g[i] * (y[i] * ry * w[i]) : x[i];
              const float p = du[i] * (x1 * rx);
              pre[v][i] += p;
              s1[0] += p * wp[i];
            }
          }
        }
        team_sum<W>(s1, red1[team], turn1, team, wit);
        m1 = s1[0] * inv_h;
      }
      float d[V][8];
      float s3[3] = {0.0f, 0.0f, 0.0f};  // sums over the row of c yn, d x and d z
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * TT + lane) * 8;
        if (col < a.H) {
          float x[8], y[8], g[8], w[8], du[8], wp[8];
          load8<DT>(a.x[rank], row + col, x);
          if (a.has_y) {
            load8<DT>(a.y[rank], row + col, y);
            load_or_one<DT>(a.w_post, col, w);
            load_gate<DT>(a, t, col, g);
          }
          if (a.has_dx_out) {
            load8<DT>(a.dx_out[rank], row + col, d[v]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[v][i] = 0.0f;
          }
          if (a.has_u) {
            load8<DT>(a.du[rank], row + col, du);
            load_or_one<DT>(a.w_pre, col, wp);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float yn = a.has_y ? y[i] * ry : 0.0f;
            const float x1 = a.has_y ? rho * x[i] + g[i] * (yn * w[i]) : x[i];
            if (a.has_u) d[v][i] += rx * (wp[i] * du[i] - x1 * rx * m1);
            if (a.has_y) {
              const float dn = d[v][i] * yn;
              if constexpr (MULTI) A[v][i] += dn;
              else post[v][i] += row_gate ? dn * g[i] : dn;
              s3[0] += dn * g[i] * w[i];
              s3[1] += d[v][i] * x[i];
              s3[2] += dn * w[i];
            }
          }
        }
      }
      float m2 = 0.0f;
      if (a.has_y) {
        team_sum<W>(s3, red3[team], turn3, team, wit);
        m2 = a.post_norm ? s3[0] * inv_h : 0.0f;
        res += s3[1];
        scalar += s3[2];
        if (row_gate && !item_scalar && a.dgate != nullptr && lane == 0) a.dgate[t] = s3[2];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * TT + lane) * 8;
        if (col < a.H) {
          if (a.has_y) {
            float y[8], g[8], w[8];
            load8<DT>(a.y[rank], row + col, y);
            load_or_one<DT>(a.w_post, col, w);
            load_gate<DT>(a, t, col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = ry * (d[v][i] * g[i] * w[i] - y[i] * ry * m2);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_b[rank]) + row + col) = pack8<DT>(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[v][i] *= rho;
          }
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_a[rank]) + row + col) = pack8<DT>(d[v]);
        }
      }
    }
    if constexpr (MULTI) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * TT + lane) * 8;
        if (col < a.H) {
          float g[8];
          load8<DT>(a.gate, static_cast<size_t>(run) * a.H + col, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) post[v][i] += g[i] * A[v][i];
        }
      }
      if (a.dgate != nullptr) {
        if (a.sub == 1) join_teams(A, a.dgate + static_cast<size_t>(run) * a.H, a.w_post);
        else join_teams(A, a.part_gate + static_cast<size_t>(item) * a.H, nullptr);
      }
    }
    if (item_scalar) join_scalar(scalar, a.part_scalar + item);
  }
  if (a.has_u) join_teams(pre, a.part_pre + static_cast<size_t>(blockIdx.x) * a.H, nullptr);
  if (a.has_y) {
    join_teams(post, a.part_post + static_cast<size_t>(blockIdx.x) * a.H, nullptr);
    join_scalar(res, a.part_res + blockIdx.x);
  }
}

constexpr int SUM_COLS = 32, SUM_WARPS = 8;

// Joins the CTAs' partial sums, each column in a fixed order, and leaves the
// partial sums zero.  blockIdx.y: 0 dw_pre, 1 dw_post (and the gradient of a
// gate of one row), 2 the scalars, 3 + g the gate row g of several.
template <int DT>
__global__ void __launch_bounds__(SUM_COLS* SUM_WARPS)
block_norm_sums_kernel(const __grid_constant__ BlockNormArgs a, int ctas, int multi) {
  __shared__ float part[SUM_WARPS][SUM_COLS];
  const int lane = threadIdx.x % SUM_COLS, warp = threadIdx.x / SUM_COLS;
  const int job = blockIdx.y;
  if (job == 2) {
    if (!a.has_y || blockIdx.x != 0) return;
    if (warp == 0) {
      double s = 0.0;
      for (int i = lane; i < ctas; i += 32) {
        s += a.part_res[i];
        a.part_res[i] = 0.0;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (a.dres != nullptr && lane == 0) a.dres[0] = static_cast<float>(s);
    }
    if (a.gate != nullptr && a.gate_cols == 1 && a.gate_per > 1) {
      for (int g = threadIdx.x; g < a.items / a.sub; g += SUM_COLS * SUM_WARPS) {
        double s = 0.0;
        for (int i = g * a.sub; i < (g + 1) * a.sub; ++i) {
          s += a.part_scalar[i];
          a.part_scalar[i] = 0.0;
        }
        if (a.dgate != nullptr) a.dgate[g] = static_cast<float>(s);
      }
    }
    return;
  }
  float* src;
  int n;
  if (job == 0) {
    if (!a.has_u) return;
    src = a.part_pre;
    n = ctas;
  } else if (job == 1) {
    if (!a.has_y) return;
    src = a.part_post;
    n = ctas;
  } else {
    src = a.part_gate + static_cast<size_t>(job - 3) * a.sub * a.H;
    n = a.sub;
  }
  const int col = blockIdx.x * SUM_COLS + lane;
  float s = 0.0f;
  if (col < a.H) {
    for (int i = warp; i < n; i += SUM_WARPS) {
      float* p = src + static_cast<size_t>(i) * a.H + col;
      s += *p;
      *p = 0.0f;
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= a.H) return;
#pragma unroll
  for (int w = 1; w < SUM_WARPS; ++w) s += part[w][lane];
  if (job == 0) {
    if (a.dw_pre != nullptr) a.dw_pre[col] = s;
    return;
  }
  const bool one_row = a.gate != nullptr && a.gate_cols != 1 && !multi;
  if (job == 1) {
    if (a.dw_post != nullptr) a.dw_post[col] = one_row ? s * load16<DT>(a.gate, col) : s;
    if (one_row && a.dgate != nullptr) a.dgate[col] = a.w_post != nullptr ? s * load16<DT>(a.w_post, col) : s;
    return;
  }
  if (a.dgate != nullptr)
    a.dgate[static_cast<size_t>(job - 3) * a.H + col] = a.w_post != nullptr ? s * load16<DT>(a.w_post, col) : s;
}

template <int N>
using Int = std::integral_constant<int, N>;

// Calls f(W, V) for the team that holds a row of H columns.
template <typename F>
flux_status_t by_width(int H, F&& f) {
  const int nvec = H / 8;
  if (nvec <= 32) return f(Int<1>{}, Int<1>{});
  if (nvec <= 64) return f(Int<1>{}, Int<2>{});
  if (nvec <= 128) return f(Int<2>{}, Int<2>{});
  if (nvec <= 256) return f(Int<4>{}, Int<2>{});
  if (nvec <= 512) return f(Int<8>{}, Int<2>{});
  if (nvec <= 1024) return f(Int<16>{}, Int<2>{});
  if (nvec <= 1536) return f(Int<16>{}, Int<3>{});
  return f(Int<16>{}, Int<4>{});
}

// How the backward pass cuts T rows into items, and its workspace.
struct BwdPlan {
  int teams, max_ctas, item_rows, sub, chunk, items, ctas;
  bool multi;
  size_t pre, post, gate, res, scalar, total;
};

BwdPlan bwd_plan(int T, int H, int gate_rows, int gate_cols) {
  BwdPlan p{};
  const int nvec = H / 8;
  p.teams = nvec <= 64 ? 8 : nvec <= 128 ? 4 : nvec <= 256 ? 2 : 1;
  p.max_ctas = nvec <= 512 ? BN_MAX_CTAS : BN_MAX_CTAS / 2;
  // several gate rows: an item stays inside one (a gate per token has its
  // gradient written row by row)
  const int per = gate_rows > 0 ? T / gate_rows : T;
  p.multi = gate_rows > 1 && gate_cols > 1;
  const bool split = gate_rows > 1 && (p.multi || per > 1);
  p.item_rows = split ? per : T;
  const int runs = split ? gate_rows : 1;
  // rounds of the grid x (rows of an item + one row's worth for its joins)
  long long best = -1;
  const int most = (p.item_rows + p.teams - 1) / p.teams;
  for (int s = 1; s <= most; ++s) {
    if (s > 1 && static_cast<long long>(runs) * s > 2 * p.max_ctas) break;
    const int chunk = (p.item_rows + s - 1) / s;
    const int sub = (p.item_rows + chunk - 1) / chunk;
    const long long items = static_cast<long long>(runs) * sub;
    const long long cost = (items + p.max_ctas - 1) / p.max_ctas * ((chunk + p.teams - 1) / p.teams + 1);
    if (best < 0 || cost < best) {
      best = cost;
      p.sub = sub;
      p.chunk = chunk;
      p.items = static_cast<int>(items);
    }
  }
  p.ctas = std::min(p.items, p.max_ctas);
  size_t at = WS_HEADER;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, WS_ALIGN);
    return here;
  };
  p.pre = take(sizeof(float) * p.ctas * H);
  p.post = take(sizeof(float) * p.ctas * H);
  p.gate = take(p.multi && p.sub > 1 ? sizeof(float) * p.items * static_cast<size_t>(H) : 0);
  p.res = take(sizeof(double) * p.ctas);
  p.scalar = take(split && !p.multi ? sizeof(double) * p.items : 0);
  p.total = at;
  return p;
}

template <typename P>
bool shards_ok(int R, P const* shards, flux_status_t* st) {
  for (int r = 0; r < R; ++r) {
    if (shards[r] == nullptr) {
      *st = FLUX_ERR_INVALID_ARG;
      return false;
    }
    if (!aligned16(shards[r])) {
      *st = FLUX_ERR_UNSUPPORTED;
      return false;
    }
  }
  return true;
}

// The rules both directions share; FLUX_OK if the call can go on.
flux_status_t check_common(int R, int T, int H, flux_dtype_t dtype, int post_norm, int gate_rows, int gate_cols,
                           bool has_y, bool has_u, const void* w_post, const void* gate, const void* res_scale,
                           const void* w_pre) {
  if (R < 1 || R > FLUX_MAX_RANKS || T < 0 || H < 0 || T % R != 0) return FLUX_ERR_INVALID_ARG;
  if (dtype != FLUX_F16 && dtype != FLUX_BF16) return FLUX_ERR_INVALID_ARG;
  if (!has_y && !has_u) return FLUX_ERR_INVALID_ARG;
  if (!has_y && (w_post != nullptr || gate != nullptr || res_scale != nullptr)) return FLUX_ERR_INVALID_ARG;
  if (has_y && !post_norm && w_post != nullptr) return FLUX_ERR_INVALID_ARG;
  if (!has_u && w_pre != nullptr) return FLUX_ERR_INVALID_ARG;
  if (gate != nullptr && (gate_rows < 1 || T % gate_rows != 0 || (gate_cols != 1 && gate_cols != H)))
    return FLUX_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > BLOCK_MAX_H) return FLUX_ERR_UNSUPPORTED;
  if (!aligned16(w_post) || !aligned16(gate) || !aligned16(res_scale) || !aligned16(w_pre)) return FLUX_ERR_UNSUPPORTED;
  return FLUX_OK;
}

void fill_common(BlockNormArgs* a, int R, int T, int H, int post_norm, int gate_rows, int gate_cols,
                 const void* const* x, const void* const* y, const void* w_post, const void* gate,
                 const float* res_scale, const void* w_pre) {
  for (int r = 0; r < R; ++r) {
    a->x[r] = x[r];
    a->y[r] = y != nullptr ? y[r] : nullptr;
  }
  a->T = T;
  a->H = H;
  a->rows_per_rank = T / R;
  a->has_y = y != nullptr;
  a->post_norm = post_norm && y != nullptr;
  a->w_post = w_post;
  a->gate = gate;
  a->gate_per = gate != nullptr ? T / gate_rows : T;
  a->gate_cols = gate != nullptr ? gate_cols : 0;
  a->res_scale = res_scale;
  a->w_pre = w_pre;
}

template <int DT>
flux_status_t launch_fwd(const BlockNormArgs& a, cudaStream_t s) {
  return by_width(a.H, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    constexpr int teams = Team<W>::COUNT;
    const int grid = static_cast<int>(std::min<long long>((a.T + teams - 1) / teams, 1 << 20));
    block_norm_kernel<DT, W, V><<<grid, Team<W>::CTA, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  });
}

template <int DT>
flux_status_t launch_bwd(const BlockNormArgs& a, const BwdPlan& p, cudaStream_t s) {
  flux_status_t st = by_width(a.H, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    if (p.multi) block_norm_bwd_kernel<DT, W, V, true><<<p.ctas, Team<W>::CTA, 0, s>>>(a);
    else block_norm_bwd_kernel<DT, W, V, false><<<p.ctas, Team<W>::CTA, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  });
  if (st != FLUX_OK) return st;
  const int rows = p.multi && p.sub > 1 && a.dgate != nullptr ? p.items / p.sub : 0;
  const dim3 grid((a.H + SUM_COLS - 1) / SUM_COLS, 3 + rows);
  block_norm_sums_kernel<DT><<<grid, SUM_COLS * SUM_WARPS, 0, s>>>(a, p.ctas, p.multi);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" flux_status_t flux_block_norm(int R, int T, int H, flux_dtype_t dtype, int post_norm, int gate_rows,
                                         int gate_cols, float eps, const void* const* x_shards,
                                         const void* const* y_shards, const void* w_post, const void* gate,
                                         const float* res_scale, const void* w_pre, void* const* x_out,
                                         void* const* u_out, float* rstd_y, float* rstd_x, void* stream) {
  flux_status_t st = check_common(R, T, H, dtype, post_norm, gate_rows, gate_cols, y_shards != nullptr,
                                  u_out != nullptr, w_post, gate, res_scale, w_pre);
  if (st != FLUX_OK) return st;
  if (!(eps >= 0.0f) || isinf(eps)) return FLUX_ERR_INVALID_ARG;
  if ((y_shards != nullptr) != (x_out != nullptr)) return FLUX_ERR_INVALID_ARG;
  if (rstd_y != nullptr && (y_shards == nullptr || !post_norm)) return FLUX_ERR_INVALID_ARG;
  if (rstd_x != nullptr && u_out == nullptr) return FLUX_ERR_INVALID_ARG;
  if (T == 0 || H == 0) return FLUX_OK;
  if (x_shards == nullptr) return FLUX_ERR_INVALID_ARG;
  if (!shards_ok(R, x_shards, &st) || (y_shards != nullptr && !shards_ok(R, y_shards, &st)) ||
      (x_out != nullptr && !shards_ok(R, x_out, &st)) || (u_out != nullptr && !shards_ok(R, u_out, &st)))
    return st;
  if (!aligned16(rstd_y) || !aligned16(rstd_x)) return FLUX_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  BlockNormArgs a{};
  fill_common(&a, R, T, H, post_norm, gate_rows, gate_cols, x_shards, y_shards, w_post, gate, res_scale, w_pre);
  a.has_u = u_out != nullptr;
  for (int r = 0; r < R; ++r) {
    a.out_a[r] = x_out != nullptr ? x_out[r] : nullptr;
    a.out_b[r] = u_out != nullptr ? u_out[r] : nullptr;
  }
  a.rstd_y = rstd_y;
  a.rstd_x = rstd_x;
  a.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == FLUX_BF16 ? launch_fwd<1>(a, s) : launch_fwd<0>(a, s);
}

extern "C" size_t flux_block_norm_workspace_size(int T, int H, int gate_rows, int gate_cols) {
  if (T < 0 || H < 0 || H % 8 != 0 || H > BLOCK_MAX_H || gate_rows < 0 || gate_cols < 0) return 0;
  if (gate_rows > 0 && gate_cols > 0 && (T % gate_rows != 0 || (gate_cols != 1 && gate_cols != H))) return 0;
  if (T == 0 || H == 0) return WS_HEADER;
  return bwd_plan(T, H, gate_cols > 0 ? gate_rows : 0, gate_cols).total;
}

extern "C" flux_status_t flux_block_norm_bwd(int R, int T, int H, flux_dtype_t dtype, int post_norm, int gate_rows,
                                             int gate_cols, const void* const* x_shards, const void* const* y_shards,
                                             const void* w_post, const void* gate, const float* res_scale,
                                             const void* w_pre, const float* rstd_y, const float* rstd_x,
                                             const void* const* dx_out, const void* const* du, void* const* dx,
                                             void* const* dy, float* dw_post, float* dgate, float* dres_scale,
                                             float* dw_pre, void* workspace, size_t workspace_bytes, void* stream) {
  flux_status_t st = check_common(R, T, H, dtype, post_norm, gate_rows, gate_cols, y_shards != nullptr,
                                  du != nullptr, w_post, gate, res_scale, w_pre);
  if (st != FLUX_OK) return st;
  const bool has_y = y_shards != nullptr;
  if (has_y != (dy != nullptr)) return FLUX_ERR_INVALID_ARG;
  // a gradient that is asked for needs what it is the gradient of
  if ((dw_post != nullptr && (!has_y || !post_norm)) || (dgate != nullptr && gate == nullptr) ||
      (dres_scale != nullptr && res_scale == nullptr) || (dw_pre != nullptr && du == nullptr))
    return FLUX_ERR_INVALID_ARG;
  if (!aligned16(rstd_y) || !aligned16(rstd_x) || !aligned16(dw_post) || !aligned16(dgate) || !aligned16(dres_scale) ||
      !aligned16(dw_pre))
    return FLUX_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0 || H == 0) {
    // sums over nothing; gate_rows divides T = 0 whatever it is
    cudaError_t e = cudaSuccess;
    auto zero = [&](float* p, size_t n) {
      if (p != nullptr && n > 0 && e == cudaSuccess) e = cudaMemsetAsync(p, 0, n * sizeof(float), s);
    };
    zero(dw_post, H);
    zero(dgate, static_cast<size_t>(gate_rows) * gate_cols);
    zero(dres_scale, 1);
    zero(dw_pre, H);
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  }
  if (x_shards == nullptr || dx == nullptr) return FLUX_ERR_INVALID_ARG;
  if ((has_y && post_norm && rstd_y == nullptr) || (du != nullptr && rstd_x == nullptr)) return FLUX_ERR_INVALID_ARG;
  if (!shards_ok(R, x_shards, &st) || (has_y && (!shards_ok(R, y_shards, &st) || !shards_ok(R, dy, &st))) ||
      (dx_out != nullptr && !shards_ok(R, dx_out, &st)) || (du != nullptr && !shards_ok(R, du, &st)) ||
      !shards_ok(R, dx, &st))
    return st;
  const BwdPlan p = bwd_plan(T, H, gate != nullptr ? gate_rows : 0, gate != nullptr ? gate_cols : 0);
  if ((st = check_workspace(workspace, workspace_bytes, p.total)) != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  BlockNormArgs a{};
  fill_common(&a, R, T, H, post_norm, gate_rows, gate_cols, x_shards, y_shards, w_post, gate, res_scale, w_pre);
  a.has_u = du != nullptr;
  a.has_dx_out = dx_out != nullptr;
  for (int r = 0; r < R; ++r) {
    a.out_a[r] = dx[r];
    a.out_b[r] = has_y ? dy[r] : nullptr;
    a.dx_out[r] = dx_out != nullptr ? dx_out[r] : nullptr;
    a.du[r] = du != nullptr ? du[r] : nullptr;
  }
  a.rstd_y = const_cast<float*>(rstd_y);
  a.rstd_x = const_cast<float*>(rstd_x);
  a.dw_post = dw_post;
  a.dgate = dgate;
  a.dres = dres_scale;
  a.dw_pre = dw_pre;
  char* ws = static_cast<char*>(workspace);
  a.part_pre = reinterpret_cast<float*>(ws + p.pre);
  a.part_post = reinterpret_cast<float*>(ws + p.post);
  a.part_gate = reinterpret_cast<float*>(ws + p.gate);
  a.part_res = reinterpret_cast<double*>(ws + p.res);
  a.part_scalar = reinterpret_cast<double*>(ws + p.scalar);
  a.items = p.items;
  a.sub = p.sub;
  a.chunk = p.chunk;
  a.item_rows = p.item_rows;
  return dtype == FLUX_BF16 ? launch_bwd<1>(a, p, s) : launch_bwd<0>(a, p, s);
}
