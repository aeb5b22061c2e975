// The edge of a block with layer norm and dropout: the block's output is dropped
// out and added to the residual stream, and the sum is normalised for the next
// block.
//
//   x' = x + drop(y)
//   u  = (x' - m) r w + b      m = mean x', r = (mean (x' - m)^2 + eps)^-1/2
//
// and, with g = w du and xn = (x' - m) r, the gradients
//
//   d  = dx' + r (g - mean g - xn mean(g xn))
//   dx = d        dy = drop(d)        dw = sum_t du xn        db = sum_t du
//
// drop(v)_i is v_i 65536 / keep where the 16 bits that belong to element i are
// below keep, else 0.  The bits are those of Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with the
// user's seed as the key and (i / 8, the user's offset) as the counter: 128 bits
// for eight neighbours, so a thread makes the bits of its own 16-byte vector and
// the backward pass makes them again instead of reading a mask.  16 bits for an
// element: p to 1 / 131072, at half the work of 32.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "flux_host.h"
#include "flux_norm.cuh"
#include "flux_rows.cuh"

namespace flux {

struct LayerNormArgs {
  const void* x[FLUX_MAX_RANKS];       // forward: x;   backward: x'
  const void* y[FLUX_MAX_RANKS];
  void* out_a[FLUX_MAX_RANKS];         // forward: x';  backward: dx
  void* out_b[FLUX_MAX_RANKS];         // forward: u;   backward: dy
  const void* dx_out[FLUX_MAX_RANKS];
  const void* du[FLUX_MAX_RANKS];
  const unsigned long long* rng;       // seed, offset
  const void* weight;
  const void* bias;
  float *mean, *rstd;
  float *dweight, *dbias;
  float *part_w, *part_b;              // backward partial sums (workspace)
  int T, H, rows_per_rank;
  int has_x, has_u, has_dx_out, has_dx, has_dy;
  int ctas;
  uint32_t keep;                       // of 65536; 65536: nothing is dropped
  float scale;                         // 65536 / keep
  float eps;
};

namespace {

// Which elements of V vectors of eight neighbours stay: the four words of each
// vector's counter, made together, so that the rounds' keys are made once.
template <int V>
struct Bits {
  uint32_t w[V][4];
};

struct Dropout {
  uint32_t k0, k1, keep, keep_high;
  unsigned long long offset;
  f32x2 scale;
  __device__ __forceinline__ Dropout(const LayerNormArgs& a, bool wanted)
      : k0(0), k1(0), keep(a.keep), keep_high(a.keep << 16), offset(0), scale(both(a.scale)) {
    if (wanted && a.keep < 65536u) {
      const unsigned long long seed = load_global(a.rng);
      k0 = static_cast<uint32_t>(seed);
      k1 = static_cast<uint32_t>(seed >> 32);
      offset = load_global(a.rng + 1);
    }
  }
  __device__ __forceinline__ bool on() const { return keep < 65536u; }
  // vectors block, block + step, ...
  template <int V>
  __device__ __forceinline__ Bits<V> draw(unsigned long long block, int step) const {
    Bits<V> b;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const unsigned long long n = block + static_cast<unsigned long long>(v) * step;
      b.w[v][0] = static_cast<uint32_t>(n);
      b.w[v][1] = static_cast<uint32_t>(n >> 32);
      b.w[v][2] = static_cast<uint32_t>(offset);
      b.w[v][3] = static_cast<uint32_t>(offset >> 32);
    }
    uint32_t k = k0, l = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const unsigned long long m0 = static_cast<unsigned long long>(b.w[v][0]) * 0xD2511F53u;
        const unsigned long long m1 = static_cast<unsigned long long>(b.w[v][2]) * 0xCD9E8D57u;
        b.w[v][0] = static_cast<uint32_t>(m1 >> 32) ^ b.w[v][1] ^ k;
        b.w[v][1] = static_cast<uint32_t>(m1);
        b.w[v][2] = static_cast<uint32_t>(m0 >> 32) ^ b.w[v][3] ^ l;
        b.w[v][3] = static_cast<uint32_t>(m0);
      }
      k += 0x9E3779B9u;
      l += 0xBB67AE85u;
    }
    return b;
  }
  // eight neighbours times scale, or zero where dropped (a NaN there too)
  __device__ __forceinline__ void apply(const uint32_t (&w)[4], f32x2 (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = halves(mul2(x[i], scale));
      // the high half is below keep where the word is below keep 2^16
      x[i] = pair((w[i] & 0xFFFFu) < keep ? h.x : 0.0f, w[i] < keep_high ? h.y : 0.0f);
    }
  }
};

// Forward.  A team of W warps walks rows, V vectors of 8 columns per thread; every
// thread copies its own columns of the rows to come into its own slots of shared
// memory and holds x' in registers from the first sum (the mean) to the second
// (of the squared distances from it: one pass over squares alone would lose the
// variance of rows with a large mean).
//
// Bound by HBM: 32768 x 4096 bf16 with a tenth dropped 174 us, 6.2 TB/s of the bytes it
// needs (issue slots 69 % busy), and as long without dropout; 2^27 elements in rows of
// 256 to 16384 columns 172 to 205 us, of 768 (a quarter of the lanes idle) 190 to 215.
// Rows of 264 to 1024 columns have three CTAs an SM: with the 64 registers of four, bf16
// spills (287 to 382 us).
template <int W, int V>
struct LnFwdShape {
  static constexpr int ROW = Team<W>::CTA * V * 32;  // bytes of two tensors' rows, all teams of the CTA
  static constexpr int DEPTH = V == 4 ? 2 : 3;
  static constexpr int SMEM = ROW * DEPTH;
  static constexpr int CTAS = W <= 2 && V == 2 ? 3 : W == 3 ? 8 : W <= 8 ? 1024 / Team<W>::CTA : V == 2 ? 2 : 1;  // per SM
};

template <int DT, int W, int V, bool HAS_Y>
__global__ void __launch_bounds__(Team<W>::CTA, (LnFwdShape<W, V>::CTAS))
layer_norm_kernel(const __grid_constant__ LayerNormArgs a) {
  constexpr int TT = Team<W>::THREADS, TEAMS = Team<W>::COUNT, CTA = Team<W>::CTA, DEPTH = LnFwdShape<W, V>::DEPTH;
  extern __shared__ uint4 ring[];  // [DEPTH][x, y][V][CTA]
  __shared__ alignas(16) float red[TEAMS][2 * W];
  const int team = threadIdx.x / TT, lane = threadIdx.x % TT, wit = lane / 32;
  int turn = 0;
  wait_for_previous();
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
          if (a.has_x) copy16_async(&slot(fill, 0, v), px + v * TT * 8);
        }
      }
      t_a = t_a > INT_MAX - step ? a.T : t_a + step;
    }
    copy_commit();
    fill = fill + 1 == DEPTH ? 0 : fill + 1;
  };
  // slots that no copy fills hold zeros: columns past H, an x not given
#pragma unroll
  for (int s = 0; s < DEPTH; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (column(v) >= a.H || !a.has_x) slot(s, 0, v) = make_uint4(0, 0, 0, 0);
      if (column(v) >= a.H) slot(s, 1, v) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) issue();
  // weight and bias as they are stored, ones and zeros where there are none
  const uint32_t one = pack2<DT>(1.0f, 1.0f);
  auto weights = [&](const void* base, uint32_t other, int v) {
    if (base == nullptr || column(v) >= a.H) return make_uint4(other, other, other, other);
    return load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + column(v)));
  };
  uint4 wq[V], bq[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    wq[v] = weights(a.weight, one, v);
    bq[v] = weights(a.bias, 0u, v);
  }
  const Dropout drop(a, HAS_Y);
  int stage = 0;
  for (long long tl = static_cast<long long>(blockIdx.x) * TEAMS + team; tl < a.T; tl += step) {
    const int t = static_cast<int>(tl);
    issue();
    const int rank = queue[0];
    const size_t row = static_cast<size_t>(t - rank * a.rows_per_rank) * a.H + lane * 8;
    copy_wait<DEPTH - 1>();
    f32x2 x1[V][4], s = 0;
    Bits<HAS_Y ? V : 1> bits = {};
    if constexpr (HAS_Y) {
      if (drop.on()) bits = drop.draw<V>(static_cast<unsigned long long>(t) * (a.H / 8) + lane, TT);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8<DT>(slot(stage, 0, v), x1[v]);
      if constexpr (HAS_Y) {
        f32x2 y[4];
        unpack8<DT>(slot(stage, 1, v), y);
        if (drop.on()) drop.apply(bits.w[v], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) x1[v][i] = add2(x1[v][i], y[i]);
        if (column(v) < a.H)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_a[rank]) + row + v * TT * 8) = pack8<DT>(x1[v]);
      }
      if (column(v) < a.H) {  // (dropout is drawn for the lanes past H too; their y is zero)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = add2(x1[v][i], s);
      }
    }
    if (a.has_u) {
      float s1[1] = {halves(s).x + halves(s).y};
      team_sum<W>(s1, red[team], turn, team, wit);
      const float mean = s1[0] * inv_h;
      const f32x2 minus = both(-mean);
      s = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x1[v][i] = add2(x1[v][i], minus);
            s = fma2(x1[v][i], x1[v][i], s);
          }
        }
      }
      s1[0] = halves(s).x + halves(s).y;
      team_sum<W>(s1, red[team], turn, team, wit);
      const float r = rsqrtf(s1[0] * inv_h + a.eps);
      if (lane == 0) {
        if (a.mean != nullptr) a.mean[t] = mean;
        if (a.rstd != nullptr) a.rstd[t] = r;
      }
      const f32x2 r2 = both(r);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          f32x2 w[4], b[4];
          unpack8<DT>(wq[v], w);
          unpack8<DT>(bq[v], b);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = fma2(mul2(x1[v][i], r2), w[i], b[i]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_b[rank]) + row + v * TT * 8) = pack8<DT>(w);
        }
      }
    }
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
  }
}

// Backward.  A CTA takes a stretch of consecutive rows, its teams one row each in
// turn, with the same slots of shared memory; both sums over a row are taken at
// once.  32768 x 4096 bf16 with a tenth dropped 226 us with the joining kernel, 5.9 TB/s
// (DRAM 75 % busy, issue slots 68 %): the weights and the column sums leave registers
// for 24 warps an SM, which wait for one another once a row.  (Rows of more than 6144 columns leave room for one CTA an SM, whose warps all
// wait for one another; more warps with fewer vectors make that worse: 16384 x 8192 with
// 32 warps of one vector 308 us, with 16 of two 249, 4061 x 12288 with 24 of two 80, with
// 16 of three 75.)  The sums of a thread's own columns over the rows (dw, db) stay in its
// registers; the teams' are joined in shared memory and the CTAs' by
// layer_norm_sums_kernel, both in a fixed order, so repeat calls give the same
// bits.
template <int W, int V>
struct LnBwdShape {
  static constexpr int ROW = Team<W>::CTA * V * 48;  // bytes of three tensors' rows, all teams of the CTA
  static constexpr int DEPTH = V == 1 ? 4 : V == 4 ? 2 : 3;
  static constexpr int JOIN = Team<W>::COUNT > 1 ? Team<W>::CTA * V * 32 : 0;
  static constexpr bool HELD = V < 4;  // the weights in registers, else in shared memory
  static constexpr int SMEM = ROW * DEPTH + JOIN + (HELD ? 0 : Team<W>::CTA * V * 16);
  static constexpr int BY_THREADS = V <= 2 && W < 16 ? 768 / Team<W>::CTA : 1, BY_SMEM = (227 << 10) / (SMEM + 1536);
  static constexpr int CTAS = BY_THREADS < BY_SMEM ? BY_THREADS : BY_SMEM;  // per SM
};

template <int DT, int W, int V, bool HAS_U>
__global__ void __launch_bounds__(Team<W>::CTA, (LnBwdShape<W, V>::CTAS))
layer_norm_bwd_kernel(const __grid_constant__ LayerNormArgs a) {
  constexpr int TT = Team<W>::THREADS, TEAMS = Team<W>::COUNT, CTA = Team<W>::CTA;
  constexpr int DEPTH = LnBwdShape<W, V>::DEPTH;
  enum { X = 0, DU = 1, DX = 2 };
  extern __shared__ uint4 ring[];  // [DEPTH][tensor][V][CTA]
  float* join = reinterpret_cast<float*>(ring + LnBwdShape<W, V>::ROW / 16 * DEPTH);
  __shared__ alignas(16) float red[TEAMS][4 * W];
  const int team = threadIdx.x / TT, lane = threadIdx.x % TT, wit = lane / 32;
  int turn = 0;
  wait_for_previous();
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const int begin = first_row(a.T, a.ctas, blockIdx.x), end = first_row(a.T, a.ctas, blockIdx.x + 1);
  auto column = [&](int v) { return (v * TT + lane) * 8; };
  auto slot = [&](int stage, int tensor, int v) -> uint4& {
    return ring[((stage * 3 + tensor) * V + v) * CTA + threadIdx.x];
  };
  struct Row {
    int rank;
    float mean, r;
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
      r.mean = HAS_U ? load_global(a.mean + t_a) : 0.0f;
      // (0 past the row's end, where (0 - m) r may be infinite although no column's n is; of
      // several vectors the sums leave those out, which would cost rows of one 8 %: 2^27
      // elements in rows of 256 with dropout 238 us, this way 224)
      r.r = HAS_U && (V > 1 || column(0) < a.H) ? load_global(a.rstd + t_a) : 0.0f;
      queue[DEPTH - 1] = r;
      const size_t at = static_cast<size_t>(t_a - rank_a * a.rows_per_rank) * a.H + lane * 8;
      const uint16_t* px = HAS_U ? static_cast<const uint16_t*>(a.x[rank_a]) + at : nullptr;
      const uint16_t* pu = HAS_U ? static_cast<const uint16_t*>(a.du[rank_a]) + at : nullptr;
      const uint16_t* pd = a.has_dx_out ? static_cast<const uint16_t*>(a.dx_out[rank_a]) + at : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          if constexpr (HAS_U) {
            copy16_async(&slot(fill, X, v), px + v * TT * 8);
            copy16_async(&slot(fill, DU, v), pu + v * TT * 8);
          }
          if (a.has_dx_out) copy16_async(&slot(fill, DX, v), pd + v * TT * 8);
        }
      }
      t_a += TEAMS;
    }
    copy_commit();
    fill = fill + 1 == DEPTH ? 0 : fill + 1;
  };
  // slots that no copy fills hold zeros: columns past H, a gradient not given
#pragma unroll
  for (int s = 0; s < DEPTH; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (column(v) >= a.H) slot(s, X, v) = slot(s, DU, v) = make_uint4(0, 0, 0, 0);
      if (column(v) >= a.H || !a.has_dx_out) slot(s, DX, v) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) issue();
  // The weights: in registers; of rows of four vectors in the thread's own places of
  // shared memory (in registers 168 bytes a thread went to local memory and back for every
  // row: 8192 x 16384 fp16 299 us).
  constexpr bool HELD = LnBwdShape<W, V>::HELD;
  const uint32_t one = pack2<DT>(1.0f, 1.0f);
  uint4 wq[HAS_U && HELD ? V : 1];
  auto weight = [&](int v) -> uint4& {
    if constexpr (HELD) return wq[v];
    else return ring[(DEPTH * 3 * V + v) * CTA + threadIdx.x];
  };
  f32x2 dw[HAS_U ? V : 1][4] = {}, db[HAS_U ? V : 1][4] = {};
  if constexpr (HAS_U) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      weight(v) = a.weight != nullptr && column(v) < a.H
                      ? load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + column(v)))
                      : make_uint4(one, one, one, one);
  }
  const Dropout drop(a, a.has_dy != 0);
  int stage = 0;
  for (int t = begin + team; t < end; t += TEAMS) {
    issue();
    const Row row = queue[0];
    copy_wait<DEPTH - 1>();
    const f32x2 minus = both(-row.mean), r2 = both(row.r);
    f32x2 k1 = 0, k2 = 0;
    if constexpr (HAS_U) {
      f32x2 sg = 0, sx = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f32x2 x[4], du[4], w[4];
        unpack8<DT>(slot(stage, X, v), x);
        unpack8<DT>(slot(stage, DU, v), du);
        unpack8<DT>(weight(v), w);
        if (V > 1 && column(v) >= a.H) continue;  // (see r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 xn = mul2(add2(x[i], minus), r2), g = mul2(du[i], w[i]);
          sg = add2(sg, g);
          sx = fma2(g, xn, sx);
          dw[v][i] = fma2(du[i], xn, dw[v][i]);
          db[v][i] = add2(db[v][i], du[i]);
        }
      }
      float s2[2] = {halves(sg).x + halves(sg).y, halves(sx).x + halves(sx).y};
      team_sum<W>(s2, red[team], turn, team, wit);
      k1 = both(-s2[0] * inv_h);
      k2 = both(-s2[1] * inv_h);
    }
    const size_t at = static_cast<size_t>(t - row.rank * a.rows_per_rank) * a.H + lane * 8;
    Bits<V> bits = {};
    if (a.has_dy && drop.on()) bits = drop.draw<V>(static_cast<unsigned long long>(t) * (a.H / 8) + lane, TT);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f32x2 d[4];
      unpack8<DT>(slot(stage, DX, v), d);
      if constexpr (HAS_U) {
        f32x2 x[4], du[4], w[4];
        unpack8<DT>(slot(stage, X, v), x);
        unpack8<DT>(slot(stage, DU, v), du);
        unpack8<DT>(weight(v), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 xn = mul2(add2(x[i], minus), r2);
          d[i] = fma2(fma2(xn, k2, add2(mul2(du[i], w[i]), k1)), r2, d[i]);
        }
      }
      if (column(v) < a.H) {
        if (a.has_dx) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_a[row.rank]) + at + v * TT * 8) = pack8<DT>(d);
        if (a.has_dy) {
          if (drop.on()) drop.apply(bits.w[v], d);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_b[row.rank]) + at + v * TT * 8) = pack8<DT>(d);
        }
      }
    }
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
  }
  if constexpr (HAS_U) {
    auto put = [&](const f32x2 (&acc)[HAS_U ? V : 1][4], float* dst) {
      auto four = [&](int v, int h) {
        const float2 lo = halves(acc[v][2 * h]), hi = halves(acc[v][2 * h + 1]);
        return make_float4(lo.x, lo.y, hi.x, hi.y);
      };
      float* own = TEAMS > 1 ? join + team * a.H : dst;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (column(v) < a.H) {
          float4* p = reinterpret_cast<float4*>(own + column(v));
          p[0] = four(v, 0);
          p[1] = four(v, 1);
        }
      }
      if constexpr (TEAMS > 1) {
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
          *reinterpret_cast<float4*>(dst + c) = s;
        }
        __syncthreads();
      }
    };
    const size_t mine = static_cast<size_t>(blockIdx.x) * a.H;
    if (a.dweight != nullptr) put(dw, a.part_w + mine);
    if (a.dbias != nullptr) put(db, a.part_b + mine);
  }
}

// Joins the CTAs' sums of dw (the first blocks) and db, and leaves them zero.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
layer_norm_sums_kernel(const __grid_constant__ LayerNormArgs a, int w_blocks) {
  __shared__ float part[WARPS][SUM_COLS];
  wait_for_previous();
  const int lane = threadIdx.x % SUM_COLS, warp = threadIdx.x / SUM_COLS;
  const bool is_w = static_cast<int>(blockIdx.x) < w_blocks;
  const int col = (is_w ? blockIdx.x : blockIdx.x - w_blocks) * SUM_COLS + lane;
  const float s = column_sum<WARPS>(is_w ? a.part_w : a.part_b, a.ctas, a.H, col, warp, lane, part);
  if (warp == 0 && col < a.H) (is_w ? a.dweight : a.dbias)[col] = s;
}

// The backward pass's grid and workspace.
struct LnPlan {
  int ctas;
  size_t w, b, total;
};

LnPlan ln_plan(int T, int H) {
  LnPlan p{};
  p.ctas = by_width<true>(H, [T](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value, TEAMS = Team<W>::COUNT;
    return std::min(LnBwdShape<W, V>::CTAS * BN_SMS, ceil_div(T, TEAMS));
  });
  const size_t each = round_up(sizeof(float) * p.ctas * H, WS_ALIGN);
  p.w = WS_HEADER;
  p.b = p.w + each;
  p.total = p.b + each;
  return p;
}

// Of 65536 draws how many keep an element; 0: p is not a share that can be dropped.
uint32_t keep_of(float p) {
  if (!(p >= 0.0f && p < 1.0f)) return 0;
  return static_cast<uint32_t>(llrint((1.0 - static_cast<double>(p)) * 65536.0));
}

template <int DT, int W, int V, bool HAS_Y>
flux_status_t launch_fwd_form(const LayerNormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  using S = LnFwdShape<W, V>;
  constexpr auto kernel = layer_norm_kernel<DT, W, V, HAS_Y>;
  const cudaError_t attr = allow_smem<kernel, S::SMEM>(dev.device);
  if (attr != cudaSuccess) return cuda_fail(attr);
  const int grid = std::min(ceil_div(a.T, Team<W>::COUNT), dev.sm_count * S::CTAS);
  const cudaError_t e = launch_behind(kernel, dim3(grid), Team<W>::CTA, S::SMEM, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int DT>
flux_status_t launch_fwd(const LayerNormArgs& a, bool has_y, const DeviceInfo& dev, cudaStream_t s) {
  return by_width<false>(a.H, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    return has_y ? launch_fwd_form<DT, W, V, true>(a, dev, s) : launch_fwd_form<DT, W, V, false>(a, dev, s);
  });
}

template <int DT, int W, int V, bool HAS_U>
flux_status_t launch_bwd_form(const LayerNormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int smem = LnBwdShape<W, V>::SMEM;
  constexpr auto kernel = layer_norm_bwd_kernel<DT, W, V, HAS_U>;
  const cudaError_t attr = allow_smem<kernel, smem>(dev.device);
  if (attr != cudaSuccess) return cuda_fail(attr);
  const cudaError_t e = launch_behind(kernel, dim3(a.ctas), Team<W>::CTA, smem, s, a);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int DT>
flux_status_t launch_bwd(const LayerNormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const flux_status_t st = by_width<true>(a.H, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    return a.has_u ? launch_bwd_form<DT, W, V, true>(a, dev, s) : launch_bwd_form<DT, W, V, false>(a, dev, s);
  });
  const int w_blocks = a.dweight != nullptr ? sum_blocks(a.H) : 0, b_blocks = a.dbias != nullptr ? sum_blocks(a.H) : 0;
  if (st != FLUX_OK || w_blocks + b_blocks == 0) return st;
  // up to 912 CTAs to join: more warps for many of them (32768 x 2048: 30 us with eight
  // warps, 9 with 32), fewer for few, where most of 32 would have nothing to add
  const cudaError_t e = a.ctas > 2 * BN_SMS ? launch_behind(layer_norm_sums_kernel<32>, dim3(w_blocks + b_blocks), 1024, 0, s, a, w_blocks)
                                            : launch_behind(layer_norm_sums_kernel<8>, dim3(w_blocks + b_blocks), 256, 0, s, a, w_blocks);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

// The rules both directions share.
flux_status_t check_common(int R, int T, int H, flux_dtype_t dtype, float p, const void* rng, const void* weight) {
  if (R < 1 || R > FLUX_MAX_RANKS || T < 0 || H < 0 || T % R != 0) return FLUX_ERR_INVALID_ARG;
  if (dtype != FLUX_F16 && dtype != FLUX_BF16) return FLUX_ERR_INVALID_ARG;
  if (keep_of(p) == 0) return FLUX_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > FLUX_BLOCK_MAX_H) return FLUX_ERR_UNSUPPORTED;
  if (!aligned16(rng) || !aligned16(weight)) return FLUX_ERR_UNSUPPORTED;
  return FLUX_OK;
}

void fill_common(LayerNormArgs* a, int R, int T, int H, float p, const void* rng, const void* weight) {
  a->T = T;
  a->H = H;
  a->rows_per_rank = T / R;
  a->keep = keep_of(p);
  a->scale = static_cast<float>(65536.0 / a->keep);
  a->rng = static_cast<const unsigned long long*>(rng);
  a->weight = weight;
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" flux_status_t flux_layer_norm(int R, int T, int H, flux_dtype_t dtype, float p, float eps,
                                         const void* const* x_shards, const void* const* y_shards,
                                         const uint64_t* rng, const void* weight, const void* bias,
                                         void* const* x_out, void* const* u_out, float* mean, float* rstd,
                                         void* stream) {
  flux_status_t st = check_common(R, T, H, dtype, p, rng, weight);
  if (st != FLUX_OK) return st;
  const bool has_y = y_shards != nullptr, has_u = u_out != nullptr;
  if (!(eps >= 0.0f) || isinf(eps)) return FLUX_ERR_INVALID_ARG;
  if (!has_y && !has_u) return FLUX_ERR_INVALID_ARG;
  if (has_y != (x_out != nullptr)) return FLUX_ERR_INVALID_ARG;
  if ((p > 0.0f) != (rng != nullptr) || (p > 0.0f && !has_y)) return FLUX_ERR_INVALID_ARG;
  if (!has_u && (weight != nullptr || bias != nullptr || mean != nullptr || rstd != nullptr)) return FLUX_ERR_INVALID_ARG;
  if (!aligned16(bias) || !aligned16(mean) || !aligned16(rstd)) return FLUX_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return FLUX_OK;
  if (x_shards == nullptr && !has_y) return FLUX_ERR_INVALID_ARG;
  if ((x_shards != nullptr && !shards_ok(R, x_shards, &st)) || (has_y && (!shards_ok(R, y_shards, &st) || !shards_ok(R, x_out, &st))) ||
      (has_u && !shards_ok(R, u_out, &st)))
    return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  LayerNormArgs a{};
  fill_common(&a, R, T, H, p, rng, weight);
  for (int r = 0; r < R; ++r) {
    a.x[r] = x_shards != nullptr ? x_shards[r] : nullptr;
    a.y[r] = has_y ? y_shards[r] : nullptr;
    a.out_a[r] = has_y ? x_out[r] : nullptr;
    a.out_b[r] = has_u ? u_out[r] : nullptr;
  }
  a.has_x = x_shards != nullptr;
  a.has_u = has_u;
  a.bias = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == FLUX_BF16 ? launch_fwd<1>(a, has_y, dev, s) : launch_fwd<0>(a, has_y, dev, s);
}

extern "C" size_t flux_layer_norm_workspace_size(int T, int H) {
  if (T < 0 || T > BWD_MAX_ROWS || H < 0 || H % 8 != 0 || H > FLUX_BLOCK_MAX_H) return 0;
  if (T == 0 || H == 0) return WS_HEADER;
  return ln_plan(T, H).total;
}

extern "C" flux_status_t flux_layer_norm_bwd(int R, int T, int H, flux_dtype_t dtype, float p,
                                             const void* const* x_out, const uint64_t* rng, const void* weight,
                                             const float* mean, const float* rstd, const void* const* dx_out,
                                             const void* const* du, void* const* dx, void* const* dy,
                                             float* dweight, float* dbias, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  flux_status_t st = check_common(R, T, H, dtype, p, rng, weight);
  if (st != FLUX_OK) return st;
  if (T > BWD_MAX_ROWS) return FLUX_ERR_UNSUPPORTED;
  const bool has_u = du != nullptr;
  if ((p > 0.0f) != (rng != nullptr)) return FLUX_ERR_INVALID_ARG;
  if (dx == nullptr && dy == nullptr) return FLUX_ERR_INVALID_ARG;
  // what belongs to a norm that the call did not have
  if (!has_u && (x_out != nullptr || weight != nullptr || mean != nullptr || rstd != nullptr || dweight != nullptr || dbias != nullptr))
    return FLUX_ERR_INVALID_ARG;
  if (!aligned16(mean) || !aligned16(rstd) || !aligned16(dweight) || !aligned16(dbias)) return FLUX_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0 || H == 0) {
    cudaError_t e = cudaSuccess;  // sums over nothing
    for (float* g : {dweight, dbias})
      if (g != nullptr && H > 0 && e == cudaSuccess) e = cudaMemsetAsync(g, 0, sizeof(float) * H, s);
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  }
  if (has_u && (x_out == nullptr || mean == nullptr || rstd == nullptr)) return FLUX_ERR_INVALID_ARG;
  if ((has_u && (!shards_ok(R, x_out, &st) || !shards_ok(R, du, &st))) || (dx_out != nullptr && !shards_ok(R, dx_out, &st)) ||
      (dx != nullptr && !shards_ok(R, dx, &st)) || (dy != nullptr && !shards_ok(R, dy, &st)))
    return st;
  const LnPlan plan = ln_plan(T, H);
  if ((st = check_workspace(workspace, workspace_bytes, plan.total)) != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  LayerNormArgs a{};
  fill_common(&a, R, T, H, p, rng, weight);
  for (int r = 0; r < R; ++r) {
    a.x[r] = has_u ? x_out[r] : nullptr;
    a.du[r] = has_u ? du[r] : nullptr;
    a.dx_out[r] = dx_out != nullptr ? dx_out[r] : nullptr;
    a.out_a[r] = dx != nullptr ? dx[r] : nullptr;
    a.out_b[r] = dy != nullptr ? dy[r] : nullptr;
  }
  a.has_u = has_u;
  a.has_dx_out = dx_out != nullptr;
  a.has_dx = dx != nullptr;
  a.has_dy = dy != nullptr;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dweight = dweight;
  a.dbias = dbias;
  a.part_w = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.w);
  a.part_b = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.b);
  a.ctas = plan.ctas;
  return dtype == FLUX_BF16 ? launch_bwd<1>(a, dev, s) : launch_bwd<0>(a, dev, s);
}
