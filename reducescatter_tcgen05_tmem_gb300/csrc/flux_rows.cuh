// Helpers of the row-wise kernels (block norms, router losses, 4-bit products):
// 16-bit vectors as floats and sums over a team of warps.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
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

// The kernels of this family are launched with launch_behind: the next one's
// blocks may come up while this one still runs (as soon as all of its own are
// there), and wait_for_previous holds them until everything that was launched
// before has finished and its writes are visible.  Every kernel starts with both.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Two fp32 values in one 64-bit register pair and the packed arithmetic on them
// (one instruction for two IEEE roundings): the row kernels spend as many issue
// slots as memory cycles without it.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight 16-bit values as four pairs, and back.
template <int DT>
__device__ __forceinline__ void unpack8(const uint4& v, f32x2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<DT>(w[i]);
    f[i] = pair(p.x, p.y);
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = halves(f[i]);
    w[i] = pack2<DT>(p.x, p.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16-byte asynchronous copies to shared memory.  The row kernels use them with
// slots that belong to one thread, so that a thread's own wait is all the
// ordering they need.
__device__ __forceinline__ void copy16_async(void* smem, const void* gmem) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// reaches after it has read this one.  16-byte aligned.
template <int W, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float* red, int& turn, int team, int warp_in_team) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (W > 1) {
    float* buf = red + turn * W * N;  // value by value, one of each warp
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[i * W + warp_in_team] = v[i];
    }
    team_sync<W>(team);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
      if constexpr (W % 4 == 0) {
#pragma unroll
        for (int w = 0; w < W; w += 4) {
          const float4 p = *reinterpret_cast<const float4*>(buf + i * W + w);
          s += (p.x + p.y) + (p.z + p.w);
        }
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) s += buf[i * W + w];
      }
      v[i] = s;
    }
  }
}

}  // namespace flux
