// Helpers of the row-wise kernels (block norms, router losses, 4-bit products):
// 16-bit vectors as floats and sums over a team of warps.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace flux {

// DT as in the GEMM kernels: 0 fp16, 1 bf16.
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (DT == 1) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == 1) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int DT>
__device__ __forceinline__ float load16(const void* p, size_t i) {
  const uint16_t v = __ldg(static_cast<const uint16_t*>(p) + i);
  if constexpr (DT == 1) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  return __half2float(__ushort_as_half(v));
}

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const float2 a = unpack2<DT>(v.x), b = unpack2<DT>(v.y), c = unpack2<DT>(v.z), d = unpack2<DT>(v.w);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Barrier of one team of W warps (teams of a CTA use ids 1, 2, ...).
template <int W>
__device__ __forceinline__ void team_sync(int team) {
  if constexpr (W == 1) {
    __syncwarp();
  } else {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
  }
}

// Sums of N values over a team of W warps, the same in every thread and in
// every run.  `red` holds 2 x W x N floats of the team; `turn` alternates
// between its halves, so one barrier per sum is enough: a half is written
// again only after the barrier of the sum in between, which every thread
// reaches after it has read this one.
template <int W, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float* red, int& turn, int team, int warp_in_team) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (W > 1) {
    float* buf = red + turn * W * N;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[warp_in_team * N + i] = v[i];
    }
    team_sync<W>(team);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = buf[i];
#pragma unroll
      for (int w = 1; w < W; ++w) s += buf[w * N + i];
      v[i] = s;
    }
  }
}

}  // namespace flux
