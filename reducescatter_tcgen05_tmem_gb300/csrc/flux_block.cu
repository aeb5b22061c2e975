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
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"
#include "flux_norm.cuh"
#include "flux_rows.cuh"

namespace flux {

constexpr int BLOCK_MAX_H = FLUX_BLOCK_MAX_H;

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
  int ctas, run_rows;  // backward: grid; rows that share one row of a gate with a gradient of its own
  float eps;
};

namespace {

// The CTA that has row t.
__host__ __device__ __forceinline__ int cta_of_row(int T, int ctas, int t) {
  return static_cast<int>(((t + 1ll) * ctas - 1) / T);
}

// Forward.  A team of W warps walks rows, V vectors of 8 columns per thread; as
// in the backward pass below every thread copies its own columns of the rows to
// come into its own slots of shared memory, and holds x' between its two sums
// in registers.  Bound by HBM: 32768 x 4096 bf16, post and pre norm, in 8 shards,
// 162 us, 6.6 TB/s.
template <int W, int V>
struct FwdShape {
  static constexpr int ROW = Team<W>::CTA * V * 32;  // bytes of two tensors' rows, all teams of the CTA
  static constexpr int DEPTH = V == 4 ? 2 : 3;
  static constexpr int SMEM = ROW * DEPTH;
  static constexpr int CTAS = W == 3 ? 8 : W <= 8 ? 1024 / Team<W>::CTA : V == 2 ? 2 : 1;  // per SM
};

template <int DT, int W, int V, bool HAS_Y>
__global__ void __launch_bounds__(Team<W>::CTA, (FwdShape<W, V>::CTAS))
block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int TT = Team<W>::THREADS, TEAMS = Team<W>::COUNT, CTA = Team<W>::CTA, DEPTH = FwdShape<W, V>::DEPTH;
  extern __shared__ uint4 ring[];  // [DEPTH][x, y][V][CTA]
  __shared__ alignas(16) float red[TEAMS][2 * W];
  const int team = threadIdx.x / TT, lane = threadIdx.x % TT, wit = lane / 32;
  int turn = 0;
  wait_for_previous();
  const float rho = a.res_scale != nullptr ? load_global(a.res_scale) : 1.0f;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const int step = gridDim.x * TEAMS;
  auto column = [&](int v) { return (v * TT + lane) * 8; };
  auto slot = [&](int stage, int tensor, int v) -> uint4& { return ring[((stage * 2 + tensor) * V + v) * CTA + threadIdx.x]; };
  int queue[DEPTH];  // the ranks of the rows on their way
  int t_a = blockIdx.x * TEAMS + team, rank_a = t_a / a.rows_per_rank, rank_end_a = (rank_a + 1) * a.rows_per_rank, fill = 0;
  auto issue = [&] {
#pragma unroll
    for (int i = 0; i + 1 < DEPTH; ++i) queue[i] = queue[i + 1];
    if (t_a < a.T) {
      while (t_a >= rank_end_a) {
        ++rank_a;
        rank_end_a += a.rows_per_rank;
      }
      queue[DEPTH - 1] = rank_a;
      const size_t at = static_cast<size_t>(t_a - rank_a * a.rows_per_rank) * a.H + lane * 8;
      const uint16_t* px = static_cast<const uint16_t*>(a.x[rank_a]) + at;
      const uint16_t* py = HAS_Y ? static_cast<const uint16_t*>(a.y[rank_a]) + at : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          if constexpr (HAS_Y) copy16_async(&slot(fill, 1, v), py + v * TT * 8);
          copy16_async(&slot(fill, 0, v), px + v * TT * 8);
        }
      }
      t_a = t_a > INT_MAX - step ? a.T : t_a + step;
    }
    copy_commit();
    fill = fill + 1 == DEPTH ? 0 : fill + 1;
  };
  // slots past H hold zeros
#pragma unroll
  for (int s = 0; s < DEPTH; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (column(v) >= a.H) slot(s, 0, v) = slot(s, 1, v) = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) issue();
  // weights as they are stored, ones where there are none
  const uint32_t one = pack2<DT>(1.0f, 1.0f);
  auto weights = [&](const void* base, size_t at, int v) {
    if (base == nullptr || column(v) >= a.H) return make_uint4(one, one, one, one);
    return load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at + column(v)));
  };
  const bool col_gate = HAS_Y && a.gate != nullptr && a.gate_cols != 1, row_gate = HAS_Y && a.gate != nullptr && a.gate_cols == 1;
  const bool one_gate = col_gate && a.gate_per == a.T;
  uint4 wq[HAS_Y ? V : 1], wp[V], gq[HAS_Y ? V : 1];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    wp[v] = weights(a.w_pre, 0, v);
    if constexpr (HAS_Y) {
      wq[v] = weights(a.w_post, 0, v);
      gq[v] = one_gate ? weights(a.gate, 0, v) : make_uint4(one, one, one, one);
    }
  }
  const f32x2 rho2 = both(rho);
  int stage = 0;
  for (long long tl = static_cast<long long>(blockIdx.x) * TEAMS + team; tl < a.T; tl += step) {
    const int t = static_cast<int>(tl);
    float g_row = 1.0f;
    if constexpr (HAS_Y) {
      if (row_gate) g_row = load16<DT>(a.gate, t / a.gate_per);
      if (col_gate && !one_gate) {
#pragma unroll
        for (int v = 0; v < V; ++v) gq[v] = weights(a.gate, static_cast<size_t>(t / a.gate_per) * a.H, v);
      }
    }
    issue();
    const int rank = queue[0];
    const size_t row = static_cast<size_t>(t - rank * a.rows_per_rank) * a.H + lane * 8;
    copy_wait<DEPTH - 1>();
    float a1 = g_row;
    if constexpr (HAS_Y) {
      if (a.post_norm) {
        f32x2 s = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          f32x2 y[4];
          unpack8<DT>(slot(stage, 1, v), y);
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fma2(y[i], y[i], s);
        }
        float s1[1] = {halves(s).x + halves(s).y};
        team_sum<W>(s1, red[team], turn, team, wit);
        const float ry = rsqrtf(s1[0] * inv_h + a.eps);
        if (lane == 0 && a.rstd_y != nullptr) a.rstd_y[t] = ry;
        a1 *= ry;
      }
    }
    // x' = rho x + g (y r_y w)
    const f32x2 a12 = both(a1);
    f32x2 x1[V][4], s = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8<DT>(slot(stage, 0, v), x1[v]);
      if constexpr (HAS_Y) {
        f32x2 y[4], w[4], g[4];
        unpack8<DT>(slot(stage, 1, v), y);
        unpack8<DT>(wq[v], w);
        unpack8<DT>(gq[v], g);
#pragma unroll
        for (int i = 0; i < 4; ++i) x1[v][i] = fma2(mul2(mul2(y[i], a12), w[i]), g[i], mul2(rho2, x1[v][i]));
        if (column(v) < a.H)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_a[rank]) + row + v * TT * 8) = pack8<DT>(x1[v]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(x1[v][i], x1[v][i], s);
    }
    if (a.has_u) {
      float s1[1] = {halves(s).x + halves(s).y};
      team_sum<W>(s1, red[team], turn, team, wit);
      const float rx = rsqrtf(s1[0] * inv_h + a.eps);
      if (lane == 0 && a.rstd_x != nullptr) a.rstd_x[t] = rx;
      const f32x2 rx2 = both(rx);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f32x2 w[4];
        unpack8<DT>(wp[v], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = mul2(mul2(x1[v][i], rx2), w[i]);
        if (column(v) < a.H)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_b[rank]) + row + v * TT * 8) = pack8<DT>(w);
      }
    }
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
  }
}

// Backward.  A CTA takes a stretch of consecutive rows, its teams one row each
// in turn.  Every thread copies its own columns of the rows to come into its
// own slots of shared memory (DEPTH rows deep, so the loads of the next rows
// run while the sums of this one meet at their barriers) and keeps the sums of
// its own columns in registers:
//   pre = sum du xn (dw_pre);
//   A   = sum g' d yn, g' the row's gate if it is one scalar, else 1.  With one
//         gate row per column for all tokens dw_post = g A and dg = w_post A; with
//         several, A is taken for each stretch of rows that share one (a run, cut
//         at the CTA's ends), which gives its share of dg and adds g A to dw_post.
// A run that lies in one CTA has its gradient written at once; shares of a run
// that several CTAs cut go to the workspace, two places for each CTA (its first
// and its last run).  The teams' sums are joined in shared memory and the CTAs'
// by block_norm_sums_kernel, both in a fixed order, so repeat calls give the
// same bits.
//
// Consecutive rows for a CTA were measured against rows dealt out in turn (T
// 32768, H 4096): 318 against 393 us.
//
// Bound by latency: the registers that hold the weights and column sums leave 12
// to 16 warps on an SM, which meet twice a row.  32768 x 4096 bf16: 312 us with
// the joining kernel, 5.2 TB/s; 4061 x 12288 f16 with 31 gate rows: 152 us, 4.0.
// Where every row or every few rows have a gate row of their own, the runs' ends
// cost more than their rows: 32768 x 4096 with as many gate rows 730 us, 131072 x
// 1024, four teams a CTA of which one works at a time, 1890 (floor 356 each); with
// a gate row for eight rows 393 and 437.
template <int W, int V>
struct BwdShape {
  static constexpr int ROW = Team<W>::CTA * V * 64;  // bytes of four tensors' rows, all teams of the CTA
  static constexpr int VECS = W * V * 32;  // of a row
  static constexpr int DEPTH = W <= 8 ? (V == 1 ? 4 : 3) : VECS <= 1024 ? 3 : VECS <= 1536 ? 2 : 1;
  static constexpr int JOIN = Team<W>::COUNT > 1 ? Team<W>::CTA * V * 32 : 0;
  static constexpr int WEIGHTS = VECS > 1536 ? VECS * 48 : VECS > 1024 ? VECS * 16 : 0;  // gw in fp32, w_pre as stored
  static constexpr int SMEM = ROW * DEPTH + JOIN + WEIGHTS;
  // per SM: with two vectors the registers of twelve warps, where eight more do not
  // make up for the spills
  static constexpr int CTAS = W > 8 ? 1 : W <= 2 || W == 8 ? 2 : 384 / Team<W>::CTA;
};

template <int DT, int W, int V, bool HAS_Y, bool HAS_U>
__global__ void __launch_bounds__(Team<W>::CTA, (BwdShape<W, V>::CTAS))
block_norm_bwd_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int TT = Team<W>::THREADS, TEAMS = Team<W>::COUNT, CTA = Team<W>::CTA;
  constexpr int DEPTH = BwdShape<W, V>::DEPTH;
  // up to 8192 columns: the weights as floats and d in registers; up to 12288:
  // w_pre in shared memory, d in two slots whose values have been used; more: all
  // weights in shared memory (reloaded from L2 they took 2/3 of the time)
  constexpr bool ROOMY = BwdShape<W, V>::VECS <= 1024, GW_REGS = BwdShape<W, V>::VECS <= 1536;
  enum { X = 0, Y = 1, DU = 2, DX = 3 };
  extern __shared__ uint4 ring[];  // [DEPTH][tensor][V][CTA]
  float* join = reinterpret_cast<float*>(ring + BwdShape<W, V>::ROW / 16 * DEPTH);
  __shared__ alignas(16) float red1[TEAMS][2 * W], red2[TEAMS][4 * W];
  __shared__ double sums[TEAMS];
  const int team = threadIdx.x / TT, lane = threadIdx.x % TT, wit = lane / 32;
  int turn1 = 0, turn2 = 0;
  wait_for_previous();
  const float rho = a.res_scale != nullptr ? load_global(a.res_scale) : 1.0f;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool row_gate = a.gate != nullptr && a.gate_cols == 1;
  const bool col_gate = a.gate != nullptr && a.gate_cols != 1;
  const bool run_scalar = row_gate && a.gate_per > 1;
  const bool runs_split = col_gate && a.gate_per < a.T;  // A per run
  const int begin = first_row(a.T, a.ctas, blockIdx.x), end = first_row(a.T, a.ctas, blockIdx.x + 1);
  f32x2 pre[V][4] = {}, A[V][4] = {};
  double res = 0.0, scalar = 0.0;  // of the team, in its first thread

  auto column = [&](int v) { return (v * TT + lane) * 8; };
  auto slot = [&](int stage, int tensor, int v) -> uint4& {
    return ring[((stage * 4 + tensor) * V + v) * CTA + threadIdx.x];
  };
  // The team's rows in order, DEPTH - 1 ahead of the one at work, each with what
  // its arithmetic needs of it.
  struct Row {
    int rank;
    float ry, rx, gt;
  };
  Row queue[DEPTH];
  int t_a = begin + team, rank_a = t_a / a.rows_per_rank, rank_end_a = (rank_a + 1) * a.rows_per_rank, fill = 0;
  auto issue = [&] {
#pragma unroll
    for (int i = 0; i + 1 < DEPTH; ++i) queue[i] = queue[i + 1];
    if (t_a < end) {
      while (t_a >= rank_end_a) {
        ++rank_a;
        rank_end_a += a.rows_per_rank;
      }
      Row r;
      r.rank = rank_a;
      r.ry = a.post_norm ? load_global(a.rstd_y + t_a) : 1.0f;
      r.rx = HAS_U ? load_global(a.rstd_x + t_a) : 0.0f;
      r.gt = row_gate ? load16<DT>(a.gate, a.gate_per == 1 ? t_a : t_a / a.gate_per) : 1.0f;
      queue[DEPTH - 1] = r;
      const size_t at = static_cast<size_t>(t_a - rank_a * a.rows_per_rank) * a.H + lane * 8;
      const uint16_t* px = static_cast<const uint16_t*>(a.x[rank_a]) + at;
      const uint16_t* py = HAS_Y ? static_cast<const uint16_t*>(a.y[rank_a]) + at : nullptr;
      const uint16_t* pu = HAS_U ? static_cast<const uint16_t*>(a.du[rank_a]) + at : nullptr;
      const uint16_t* pd = a.has_dx_out ? static_cast<const uint16_t*>(a.dx_out[rank_a]) + at : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          copy16_async(&slot(fill, X, v), px + v * TT * 8);
          if constexpr (HAS_Y) copy16_async(&slot(fill, Y, v), py + v * TT * 8);
          if constexpr (HAS_U) copy16_async(&slot(fill, DU, v), pu + v * TT * 8);
          if (a.has_dx_out) copy16_async(&slot(fill, DX, v), pd + v * TT * 8);
        }
      }
      t_a += TEAMS;
    }
    copy_commit();
    fill = fill + 1 == DEPTH ? 0 : fill + 1;
  };

  // the product of w_post and the gate's columns, and w_pre
  f32x2 gw_r[GW_REGS ? V : 1][4], wp_r[ROOMY ? V : 1][4];
  uint4* gw_s = reinterpret_cast<uint4*>(join);  // [2][V][CTA] if not in registers, then w_pre [V][CTA] (JOIN is 0 there)
  uint4* wp_s = gw_s + (GW_REGS ? 0 : 2 * V * CTA);
  const uint32_t one16 = pack2<DT>(1.0f, 1.0f);
  auto weight8 = [&](const void* base, size_t at, bool inside, f32x2 (&f)[4]) {
    if (!inside) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = 0;
    } else if (base != nullptr) {
      unpack8<DT>(load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at)), f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = both(1.0f);
    }
  };
  auto load_gw = [&](int v, int run, f32x2 (&gw)[4]) {
    const bool inside = column(v) < a.H;
    weight8(a.w_post, column(v), inside, gw);
    if (col_gate) {
      f32x2 g[4];
      weight8(a.gate, static_cast<size_t>(run) * a.H + column(v), inside, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) gw[i] = mul2(gw[i], g[i]);
    }
  };
  auto put_gw = [&](int run) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (GW_REGS) {
        load_gw(v, run, gw_r[v]);
      } else {
        f32x2 gw[4];
        load_gw(v, run, gw);
        const ulonglong2 lo = make_ulonglong2(gw[0], gw[1]), hi = make_ulonglong2(gw[2], gw[3]);
        gw_s[v * CTA + threadIdx.x] = *reinterpret_cast<const uint4*>(&lo);
        gw_s[(V + v) * CTA + threadIdx.x] = *reinterpret_cast<const uint4*>(&hi);
      }
    }
  };
  auto get_gw = [&](int v, f32x2 (&gw)[4]) {
    if constexpr (GW_REGS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) gw[i] = gw_r[v][i];
    } else {
      const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(gw_s + v * CTA + threadIdx.x);
      const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(gw_s + (V + v) * CTA + threadIdx.x);
      gw[0] = lo.x, gw[1] = lo.y, gw[2] = hi.x, gw[3] = hi.y;
    }
  };
  auto get_wp = [&](int v, f32x2 (&wp)[4]) {
    if constexpr (ROOMY) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wp[i] = wp_r[v][i];
    } else {
      unpack8<DT>(wp_s[v * CTA + threadIdx.x], wp);
    }
  };
  if constexpr (HAS_U) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (column(v) < a.H)
        q = a.w_pre != nullptr
                ? load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w_pre) + column(v)))
                : make_uint4(one16, one16, one16, one16);
      if constexpr (ROOMY) unpack8<DT>(q, wp_r[v]);
      else wp_s[v * CTA + threadIdx.x] = q;
    }
  }

  // f(column, sum over teams) for every column, four at a time
  auto join_teams = [&](const f32x2 (&acc)[V][4], auto&& f) {
    auto four = [&](int v, int h) {
      const float2 lo = halves(acc[v][2 * h]), hi = halves(acc[v][2 * h + 1]);
      return make_float4(lo.x, lo.y, hi.x, hi.y);
    };
    if constexpr (TEAMS > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          float4* p = reinterpret_cast<float4*>(join + team * a.H + column(v));
          p[0] = four(v, 0);
          p[1] = four(v, 1);
        }
      }
      __syncthreads();
      for (int c = threadIdx.x * 4; c < a.H; c += CTA * 4) {
        float4 s = *reinterpret_cast<const float4*>(join + c);
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) {
          const float4 o = *reinterpret_cast<const float4*>(join + k * a.H + c);
          s.x += o.x;
          s.y += o.y;
          s.z += o.z;
          s.w += o.w;
        }
        f(c, s);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          f(column(v), four(v, 0));
          f(column(v) + 4, four(v, 1));
        }
      }
    }
  };
  auto times = [&](const void* w, size_t at, float4 s) {
    if (w != nullptr) {
      const uint2 p = load_global(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + at));
      const float2 lo = unpack2<DT>(p.x), hi = unpack2<DT>(p.y);
      s.x *= lo.x;
      s.y *= lo.y;
      s.z *= hi.x;
      s.w *= hi.y;
    }
    return s;
  };
  auto join_scalar = [&](double v) {
    if (lane == 0) sums[team] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0) {
      s = sums[0];
      for (int k = 1; k < TEAMS; ++k) s += sums[k];
    }
    __syncthreads();
    return s;
  };
  float* my_post = a.part_post + static_cast<size_t>(blockIdx.x) * a.H;
  float* my_pre = a.part_pre + static_cast<size_t>(blockIdx.x) * a.H;
  const f32x2 rho2 = both(rho);

  // slots that no copy fills hold zeros: columns past H, a gradient not given
#pragma unroll
  for (int s = 0; s < DEPTH; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (column(v) >= a.H) slot(s, X, v) = slot(s, Y, v) = slot(s, DU, v) = make_uint4(0, 0, 0, 0);
      if (column(v) >= a.H || !a.has_dx_out) slot(s, DX, v) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) issue();
  int stage = 0, t = begin + team;
  for (int t0 = begin, t1; t0 < end; t0 = t1) {
    const int run = t0 / a.run_rows;
    t1 = min(end, (run + 1) * a.run_rows);
    const bool whole = t0 == run * a.run_rows && t1 == (run + 1) * a.run_rows;
    const size_t place = 2 * blockIdx.x + (t0 == begin ? 0 : 1);  // of a cut run
    if constexpr (HAS_Y) put_gw(run);
    for (; t < t1; t += TEAMS) {
      issue();
      const Row r = queue[0];
      copy_wait<DEPTH - 1>();
      const float a1 = r.ry * r.gt;
      const f32x2 a12 = both(a1);
      // x' = rho x + y a1 gw
      float m1 = 0.0f;
      const f32x2 rx2 = both(r.rx);
      if constexpr (HAS_U) {
        f32x2 s = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          f32x2 x[4], du[4], wp[4];
          unpack8<DT>(slot(stage, X, v), x);
          unpack8<DT>(slot(stage, DU, v), du);
          get_wp(v, wp);
          if constexpr (HAS_Y) {
            f32x2 y[4], gw[4];
            unpack8<DT>(slot(stage, Y, v), y);
            get_gw(v, gw);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = fma2(mul2(y[i], a12), gw[i], mul2(rho2, x[i]));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x2 p = mul2(du[i], mul2(x[i], rx2));
            pre[v][i] = add2(pre[v][i], p);
            s = fma2(p, wp[i], s);
          }
        }
        float s1[1] = {halves(s).x + halves(s).y};
        team_sum<W>(s1, red1[team], turn1, team, wit);
        m1 = s1[0] * inv_h;
      }
      const f32x2 k1 = both(-r.rx * r.rx * m1);
      f32x2 d_r[ROOMY ? V : 1][4];
      f32x2 sy = 0, sx = 0;  // sums over the row of d y gw and d x
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f32x2 x[4], y[4], d[4], gw[4];
        unpack8<DT>(slot(stage, X, v), x);
        unpack8<DT>(slot(stage, DX, v), d);
        if constexpr (HAS_Y) {
          unpack8<DT>(slot(stage, Y, v), y);
          get_gw(v, gw);
        }
        if constexpr (HAS_U) {
          f32x2 du[4], wp[4];
          unpack8<DT>(slot(stage, DU, v), du);
          get_wp(v, wp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x2 x1 = x[i];
            if constexpr (HAS_Y) x1 = fma2(mul2(y[i], a12), gw[i], mul2(rho2, x[i]));
            d[i] = fma2(x1, k1, fma2(mul2(wp[i], du[i]), rx2, d[i]));
          }
        }
        if constexpr (HAS_Y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x2 e = mul2(d[i], y[i]);
            A[v][i] = fma2(e, a12, A[v][i]);
            sy = fma2(e, gw[i], sy);
            sx = fma2(d[i], x[i], sx);
          }
        }
        if constexpr (ROOMY) {
#pragma unroll
          for (int i = 0; i < 4; ++i) d_r[v][i] = d[i];
        } else if (column(v) < a.H) {
          // slots past H stay zero: no copy fills them again, and there d of a row that
          // is not finite is NaN
          const ulonglong2 lo = make_ulonglong2(d[0], d[1]), hi = make_ulonglong2(d[2], d[3]);
          slot(stage, X, v) = *reinterpret_cast<const uint4*>(&lo);
          slot(stage, DU, v) = *reinterpret_cast<const uint4*>(&hi);
        }
      }
      float k2 = 0.0f;
      if constexpr (HAS_Y) {
        float s2[2] = {halves(sy).x + halves(sy).y, halves(sx).x + halves(sx).y};
        team_sum<W>(s2, red2[team], turn2, team, wit);
        k2 = a.post_norm ? r.ry * r.ry * a1 * s2[0] * inv_h : 0.0f;
        if (lane == 0) {
          res += s2[1];
          if (row_gate) {
            const float dg = r.ry * s2[0];
            scalar += dg;
            if (!run_scalar && a.dgate != nullptr) a.dgate[t] = dg;
          }
        }
      }
      const f32x2 nk2 = both(-k2);
      const size_t at = static_cast<size_t>(t - r.rank * a.rows_per_rank) * a.H + lane * 8;
      uint16_t* pdx = static_cast<uint16_t*>(a.out_a[r.rank]) + at;
      uint16_t* pdy = HAS_Y ? static_cast<uint16_t*>(a.out_b[r.rank]) + at : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f32x2 d[4];
        if constexpr (ROOMY) {
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = d_r[v][i];
        } else {
          const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(&slot(stage, X, v));
          const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(&slot(stage, DU, v));
          d[0] = lo.x, d[1] = lo.y, d[2] = hi.x, d[3] = hi.y;
        }
        if constexpr (HAS_Y) {
          f32x2 y[4], gw[4];
          unpack8<DT>(slot(stage, Y, v), y);
          get_gw(v, gw);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = fma2(mul2(d[i], a12), gw[i], mul2(y[i], nk2));
            d[i] = mul2(d[i], rho2);
          }
          if (column(v) < a.H) *reinterpret_cast<uint4*>(pdy + v * TT * 8) = pack8<DT>(y);
        }
        if (column(v) < a.H) *reinterpret_cast<uint4*>(pdx + v * TT * 8) = pack8<DT>(d);
      }
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
    }
    if (runs_split) {
      const size_t grow = static_cast<size_t>(run) * a.H;
      join_teams(A, [&](int c, float4 s) {
        if (a.dgate != nullptr) {
          if (whole) *reinterpret_cast<float4*>(a.dgate + grow + c) = times(a.w_post, c, s);
          else *reinterpret_cast<float4*>(a.part_gate + place * a.H + c) = s;
        }
        // the same thread holds these columns in every run
        s = times(a.gate, grow + c, s);
        if (t0 != begin) {
          const float4 o = *reinterpret_cast<const float4*>(my_post + c);
          s.x += o.x;
          s.y += o.y;
          s.z += o.z;
          s.w += o.w;
        }
        *reinterpret_cast<float4*>(my_post + c) = s;
      });
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) A[v][i] = 0;
    }
    if (run_scalar) {
      const double s = join_scalar(scalar);
      if (threadIdx.x == 0 && a.dgate != nullptr) {
        if (whole) a.dgate[run] = static_cast<float>(s);
        else a.part_scalar[place] = s;
      }
      scalar = 0.0;
    }
  }
  if constexpr (HAS_U) join_teams(pre, [&](int c, float4 s) { *reinterpret_cast<float4*>(my_pre + c) = s; });
  if constexpr (HAS_Y) {
    if (!runs_split) join_teams(A, [&](int c, float4 s) { *reinterpret_cast<float4*>(my_post + c) = s; });
    const double s = join_scalar(res);
    if (threadIdx.x == 0) a.part_res[blockIdx.x] = s;
  }
}

// blocks of block_norm_sums_kernel: dw_pre and dw_post by columns, the scalars, cut runs by columns
inline int run_blocks(int H) { return (H + 4 * SUM_THREADS - 1) / (4 * SUM_THREADS); }

// Joins the CTAs' partial sums, each column in a fixed order, and leaves the
// partial sums zero (H 4096, 304 CTAs: 16 us with cold caches).
template <int DT>
__global__ void __launch_bounds__(SUM_THREADS)
block_norm_sums_kernel(const __grid_constant__ BlockNormArgs a, int col_blocks, int per_run_blocks) {
  __shared__ float part[SUM_WARPS][SUM_COLS];
  wait_for_previous();
  const int lane = threadIdx.x % SUM_COLS, warp = threadIdx.x / SUM_COLS;
  const bool one_row = a.gate != nullptr && a.gate_cols != 1 && a.gate_per == a.T;
  if (blockIdx.x < 2 * col_blocks) {
    const bool is_pre = blockIdx.x < col_blocks;
    if (is_pre ? !a.has_u : !a.has_y) return;
    float* src = is_pre ? a.part_pre : a.part_post;
    const int col = (is_pre ? blockIdx.x : blockIdx.x - col_blocks) * SUM_COLS + lane;
    const float s = column_sum(src, a.ctas, a.H, col, warp, lane, part);
    if (warp != 0 || col >= a.H) return;
    if (is_pre) {
      if (a.dw_pre != nullptr) a.dw_pre[col] = s;
    } else {
      if (a.dw_post != nullptr) a.dw_post[col] = one_row ? s * load16<DT>(a.gate, col) : s;
      if (one_row && a.dgate != nullptr) a.dgate[col] = a.w_post != nullptr ? s * load16<DT>(a.w_post, col) : s;
    }
    return;
  }
  if (blockIdx.x == 2 * col_blocks) {
    if (!a.has_y || warp != 0) return;
    double s = 0.0;
    for (int i = lane; i < a.ctas; i += 32) {
      s += a.part_res[i];
      a.part_res[i] = 0.0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (a.dres != nullptr && lane == 0) a.dres[0] = static_cast<float>(s);
    return;
  }
  // the run that CTA b - 1 and CTA b share, if b is the first to continue it
  const int k = blockIdx.x - 2 * col_blocks - 1;
  __shared__ int run_s, first_s, c0_s, c1_s;
  if (threadIdx.x == 0) {
    const int b = 1 + k / per_run_blocks, at = first_row(a.T, a.ctas, b), r = at / a.run_rows, r0 = r * a.run_rows;
    run_s = r;
    c0_s = cta_of_row(a.T, a.ctas, r0);
    c1_s = r0 == at || c0_s != b - 1 ? -1 : cta_of_row(a.T, a.ctas, r0 + a.run_rows - 1);
    first_s = 2 * c0_s + (first_row(a.T, a.ctas, c0_s) == r0 ? 0 : 1);
  }
  __syncthreads();
  const int run = run_s, first = first_s, c0 = c0_s, c1 = c1_s;
  if (c1 < 0) return;
  auto place = [&](int i) { return i == 0 ? first : 2 * (c0 + i); };
  const int n = c1 - c0 + 1;
  constexpr int RUN_BATCH = 8;
  if (a.gate_cols == 1) {
    if (threadIdx.x != 0 || k % per_run_blocks != 0) return;
    double s = 0.0;
    for (int i = 0; i < n; ++i) {
      s += a.part_scalar[place(i)];
      a.part_scalar[place(i)] = 0.0;
    }
    a.dgate[run] = static_cast<float>(s);
    return;
  }
  const int col = (k % per_run_blocks * SUM_THREADS + threadIdx.x) * 4;
  if (col >= a.H) return;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = 0; i0 < n; i0 += RUN_BATCH) {
    float4 v[RUN_BATCH];
#pragma unroll
    for (int j = 0; j < RUN_BATCH; ++j)
      if (i0 + j < n) v[j] = *reinterpret_cast<const float4*>(a.part_gate + static_cast<size_t>(place(i0 + j)) * a.H + col);
#pragma unroll
    for (int j = 0; j < RUN_BATCH; ++j) {
      if (i0 + j >= n) break;
      *reinterpret_cast<float4*>(a.part_gate + static_cast<size_t>(place(i0 + j)) * a.H + col) =
          make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      s.x += v[j].x;
      s.y += v[j].y;
      s.z += v[j].z;
      s.w += v[j].w;
    }
  }
  if (a.w_post != nullptr) {
    s.x *= load16<DT>(a.w_post, col);
    s.y *= load16<DT>(a.w_post, col + 1);
    s.z *= load16<DT>(a.w_post, col + 2);
    s.w *= load16<DT>(a.w_post, col + 3);
  }
  *reinterpret_cast<float4*>(a.dgate + static_cast<size_t>(run) * a.H + col) = s;
}

// The backward pass's grid and workspace.
struct BwdPlan {
  int ctas, run_rows;
  bool cut_runs;  // several gate rows with a gradient of their own (not one written token by token)
  size_t pre, post, gate, res, scalar, total;
};

BwdPlan bwd_plan(int T, int H, int gate_rows, int gate_cols) {
  BwdPlan p{};
  p.ctas = by_width<true>(H, [T](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value, TEAMS = Team<W>::COUNT;
    return std::min(BwdShape<W, V>::CTAS * BN_SMS, (T + TEAMS - 1) / TEAMS);
  });
  const int per = gate_rows > 0 ? T / gate_rows : T;
  const bool rows = gate_rows > 1 && gate_cols > 1, scalars = gate_cols == 1 && per > 1;
  p.cut_runs = rows || scalars;
  p.run_rows = p.cut_runs ? per : T;
  size_t at = WS_HEADER;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, WS_ALIGN);
    return here;
  };
  p.pre = take(sizeof(float) * p.ctas * H);
  p.post = take(sizeof(float) * p.ctas * H);
  p.gate = take(rows ? sizeof(float) * 2 * p.ctas * H : 0);
  p.res = take(sizeof(double) * p.ctas);
  p.scalar = take(scalars ? sizeof(double) * 2 * p.ctas : 0);
  p.total = at;
  return p;
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

template <int DT, int W, int V, bool HAS_Y>
flux_status_t launch_fwd_form(const BlockNormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  using S = FwdShape<W, V>;
  constexpr auto kernel = block_norm_kernel<DT, W, V, HAS_Y>;
  const cudaError_t attr = allow_smem<kernel, S::SMEM>(dev.device);
  if (attr != cudaSuccess) return cuda_fail(attr);
  const int grid = std::min(ceil_div(a.T, Team<W>::COUNT), dev.sm_count * S::CTAS);
  const cudaError_t e = launch_behind(kernel, dim3(grid), Team<W>::CTA, S::SMEM, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int DT>
flux_status_t launch_fwd(const BlockNormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  return by_width<false>(a.H, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    return a.has_y ? launch_fwd_form<DT, W, V, true>(a, dev, s) : launch_fwd_form<DT, W, V, false>(a, dev, s);
  });
}

template <int DT, int W, int V, bool HAS_Y, bool HAS_U>
flux_status_t launch_bwd_form(const BlockNormArgs& a, const BwdPlan& p, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int smem = BwdShape<W, V>::SMEM;
  constexpr auto kernel = block_norm_bwd_kernel<DT, W, V, HAS_Y, HAS_U>;
  const cudaError_t attr = allow_smem<kernel, smem>(dev.device);
  if (attr != cudaSuccess) return cuda_fail(attr);
  const cudaError_t e = launch_behind(kernel, dim3(p.ctas), Team<W>::CTA, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int DT>
flux_status_t launch_bwd(const BlockNormArgs& a, const BwdPlan& p, const DeviceInfo& dev, cudaStream_t s) {
  flux_status_t st = by_width<true>(a.H, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    if (!a.has_y) return launch_bwd_form<DT, W, V, false, true>(a, p, dev, s);
    return a.has_u ? launch_bwd_form<DT, W, V, true, true>(a, p, dev, s) : launch_bwd_form<DT, W, V, true, false>(a, p, dev, s);
  });
  if (st != FLUX_OK) return st;
  const int cols = sum_blocks(a.H), per_run = a.gate_cols == 1 ? 1 : run_blocks(a.H);
  const int cut = p.cut_runs && a.dgate != nullptr ? (p.ctas - 1) * per_run : 0;
  const cudaError_t e = launch_behind(block_norm_sums_kernel<DT>, dim3(2 * cols + 1 + cut), SUM_THREADS, 0, s, a, cols, per_run);
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
  return dtype == FLUX_BF16 ? launch_fwd<1>(a, dev, s) : launch_fwd<0>(a, dev, s);
}

extern "C" size_t flux_block_norm_workspace_size(int T, int H, int gate_rows, int gate_cols) {
  if (T < 0 || T > BWD_MAX_ROWS || H < 0 || H % 8 != 0 || H > BLOCK_MAX_H || gate_rows < 0 || gate_cols < 0) return 0;
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
  if (T > BWD_MAX_ROWS) return FLUX_ERR_UNSUPPORTED;
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
  a.ctas = p.ctas;
  a.run_rows = p.run_rows;
  return dtype == FLUX_BF16 ? launch_bwd<1>(a, p, dev, s) : launch_bwd<0>(a, p, dev, s);
}
