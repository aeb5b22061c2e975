// What the norm kernels (block norm, layer norm) share: teams of warps that hold a
// row, the choice of a team by the row's width, checks of the row shards.
#pragma once

#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "flux_host.h"

namespace flux {

constexpr int BN_SMS = 152;  // the backward grids: one wave on them
constexpr int BWD_MAX_ROWS = INT_MAX - 511;  // the backward passes count rows in ints up to the teams of a CTA past the last one

// A row is held by a team of W warps; a CTA has one to eight teams.  Where a team
// has three warps or more, CTAs of one team are faster than CTAs of several
// (2^27 elements in rows of 1792: backward 278 us, two teams 339; forward 164, 212).
template <int W>
struct Team {
  static constexpr int THREADS = W * 32;
  static constexpr int CTA = W <= 2 ? 256 : W * 32;
  static constexpr int COUNT = CTA / THREADS;
};

// CTA c of `ctas` takes the rows [first_row(c), first_row(c + 1)).
__host__ __device__ __forceinline__ int first_row(int T, int ctas, int c) {
  return static_cast<int>(static_cast<long long>(c) * T / ctas);
}

template <int N>
using Int = std::integral_constant<int, N>;

// Calls f(W, V) for the team that holds a row of H columns.  From 1032 columns on
// the steps are close enough that a third of the lanes idle at most (2^27 elements
// in rows of 5120: backward 353 us, in teams of 16 warps 401; of 1280: 278, 4 warps
// 399; of 2560: 287, 8 warps 373); just past 256 and 512 columns half of them do.
// A warp with two vectors is fast enough forward but spills backward (H 512: 456
// us, two warps of one vector 266).
template <bool BACKWARD, typename F>
auto by_width(int H, F&& f) {
  const int nvec = H / 8;
  if (nvec <= 32) return f(Int<1>{}, Int<1>{});
  if (nvec <= 64) {
    if constexpr (BACKWARD) return f(Int<2>{}, Int<1>{});
    else return f(Int<1>{}, Int<2>{});
  }
  if (nvec <= 128) return f(Int<2>{}, Int<2>{});
  if (nvec <= 192) return f(Int<3>{}, Int<2>{});
  if (nvec <= 256) return f(Int<4>{}, Int<2>{});
  if (nvec <= 384) return f(Int<6>{}, Int<2>{});
  if (nvec <= 512) return f(Int<8>{}, Int<2>{});
  if (nvec <= 768) return f(Int<12>{}, Int<2>{});
  if (nvec <= 1024) return f(Int<16>{}, Int<2>{});
  if (nvec <= 1536) return f(Int<16>{}, Int<3>{});
  return f(Int<16>{}, Int<4>{});
}

template <typename P>
inline bool shards_ok(int R, P const* shards, flux_status_t* st) {
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

// Sums over the CTAs' partial sums [ctas x H] of one column, by blocks of
// SUM_COLS columns x WARPS warps, in a fixed order; leaves the partial sums
// zero.  The sum is in the lanes of warp 0; every thread of the block calls this.
// SUM_BATCH loads of a thread are on their way together: a few MB from L2 are
// bound by latency (one load after the other, each behind the store of the last,
// took 300 us where this takes 16).
constexpr int SUM_COLS = 32, SUM_WARPS = 8, SUM_BATCH = 20, SUM_THREADS = SUM_COLS * SUM_WARPS;
inline int sum_blocks(int H) { return (H + SUM_COLS - 1) / SUM_COLS; }

template <int WARPS>
__device__ __forceinline__ float column_sum(float* src, int ctas, int H, int col, int warp, int lane,
                                            float (&part)[WARPS][SUM_COLS]) {
  float s = 0.0f;
  if (col < H) {
    for (int i0 = warp; i0 < ctas; i0 += WARPS * SUM_BATCH) {
      float v[SUM_BATCH];
#pragma unroll
      for (int j = 0; j < SUM_BATCH; ++j) {
        const int i = i0 + j * WARPS;
        v[j] = i < ctas ? src[static_cast<size_t>(i) * H + col] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < SUM_BATCH; ++j) {
        const int i = i0 + j * WARPS;
        if (i < ctas) src[static_cast<size_t>(i) * H + col] = 0.0f;
        s += v[j];
      }
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < WARPS; ++w) s += part[w][lane];
  }
  return s;
}

// Lets a kernel use SMEM bytes of shared memory, once on each device.
template <auto KERNEL, int SMEM>
cudaError_t allow_smem(int device) {
  static OncePerDevice once;
  return once(device, [] { return cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
}

}  // namespace flux
