// Products in 8-bit integers: rows quantised as they come, and
//
//   out[m, n] = x_scale[m] w_scale[n] sum_k x[m, k] w[n, k]  (+ bias[n])
//
// with integer codes x [M x K] and w [N x K].
//
// Few rows are bound by the weights' bytes: they go from HBM straight into the
// registers of 8-bit tensor-core instructions, whose integer sums are exact in any
// order.  Many rows are bound by the tensor cores, whose 8-bit integer rate on
// this GPU is a fraction of the 16-bit one; flux_q8_gemm.cu widens the codes to
// fp16, which holds them exactly, and uses that.
#include <math.h>

#include <algorithm>

#include "flux_q8.h"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int Q8_SMS = 152;
constexpr int Q8_MAX_K = 131072 - 16;  // 2^14 K stays within 32 bits

// ---------------------------------------------------------------- quantisation

constexpr int QZ_VECS = 4;  // vectors of 8 that a thread holds of a row

// scale = largest magnitude / 127 in fp32, code = x / scale to the nearest, ties to
// even.  The quotient is that of the real numbers: where the remainder x - code scale
// is next to half a scale, the fp32 estimate is corrected by it.  A fused multiply-add
// gives the remainder exactly (x has 11 bits, the code 7, the scale 24, and the
// remainder is below the scale).  One element in 30000 is that close; to correct every
// one took twice the time.  4096 x 4096 11 us, 4.6 TB/s: half of the issue slots.
// A row that holds a NaN or an infinity gets such a scale and codes of zero.
template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS)
q8_quantize_kernel(const void* x, int8_t* q, float* scales, int K) {
  __shared__ uint32_t red[THREADS / 32];
  wait_for_previous();
  const size_t at = static_cast<size_t>(blockIdx.x) * K;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
  const int nvec = K / 8;
  uint4 held[QZ_VECS];
  uint32_t top = 0;  // two 16-bit magnitudes: their bits order them, a NaN above all
  auto see = [&](const uint4& v) {
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  };
#pragma unroll
  for (int i = 0; i < QZ_VECS; ++i) {
    const int v = i * THREADS + threadIdx.x;
    held[i] = v < nvec ? load_global(src + v) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < QZ_VECS; ++i) see(held[i]);
  for (int v = QZ_VECS * THREADS + threadIdx.x; v < nvec; v += THREADS) see(load_global(src + v));
  top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) top = max(top, red[w]);
  const float amax = unpack2<DT>(top).x;
  const float scale = __fdiv_rn(amax, 127.0f), inv = __fdiv_rn(1.0f, scale);
  const bool plain = scale > 0x1p-120f && amax < INFINITY;  // v inv is v / scale to 2^-23 of it
  // the code beside an estimate of it
  auto exact = [&](float v, float c) {
    if (!plain) c = amax < INFINITY && amax > 0.0f ? rintf(__fdiv_rn(v, scale)) : 0.0f;
    const float twice = 2.0f * fmaf(-c, scale, v);
    const bool odd = (static_cast<int>(c) & 1) != 0;
    if (twice > scale || (twice == scale && odd)) c += 1.0f;
    if (twice < -scale || (twice == -scale && odd)) c -= 1.0f;
    return static_cast<uint32_t>(static_cast<int>(c));
  };
  constexpr float SHIFT = 12582912.0f;  // 1.5 2^23: a sum with it is a whole number, the low byte its code
  const float half = 0.5f * scale, margin = 0x1p-15f * scale;
  uint2* dst = reinterpret_cast<uint2*>(q + at);
  auto put = [&](int v, const uint4& u) {
    float f[8];
    unpack8<DT>(u, f);
    uint32_t c[8];
    bool close = !plain;  // a remainder next to half a scale: the estimate may be the neighbour of the code
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float shifted = fmaf(f[i], inv, SHIFT);
      c[i] = __float_as_uint(shifted);
      const float rest = fmaf(-(shifted - SHIFT), scale, f[i]);
      close |= fabsf(fabsf(rest) - half) <= margin;
    }
    if (close) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = exact(f[i], __uint_as_float(c[i]) - SHIFT);
    }
    auto four = [&](int i) {
      return __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
    };
    dst[v] = make_uint2(four(0), four(4));
  };
#pragma unroll
  for (int i = 0; i < QZ_VECS; ++i) {
    const int v = i * THREADS + threadIdx.x;
    if (v < nvec) put(v, held[i]);
  }
  for (int v = QZ_VECS * THREADS + threadIdx.x; v < nvec; v += THREADS) put(v, load_global(src + v));
  if (threadIdx.x == 0) scales[blockIdx.x] = scale;
}

// ---------------------------------------------------------------- few rows

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int FEW_ROWS = 8;             // of x: the columns of one instruction
constexpr int FEW_WARPS = 8, FEW_THREADS = FEW_WARPS * 32, FEW_CTAS = 3;
constexpr int FEW_CH = 16;              // channels of a block: the rows of one instruction
constexpr int FEW_K = FEW_WARPS * 128;  // of a step: 128 codes a warp
constexpr int FEW_DEPTH = 2;            // steps on their way
constexpr int FEW_SLOT = FEW_ROWS * FEW_CH;

struct FewPlan {
  int blocks, steps;  // of channels; of K in a block
  int ctas;           // as many as blocks: each has one; else equal stretches of steps
  size_t total;       // bytes past the header
};

// Whole blocks leave some SMs idle at the end, equal stretches need the parts of cut
// blocks joined by a second kernel, which costs about as much as 6 steps (4096 x 4096: 7
// steps an SM on average, 8 with whole blocks, which are faster by 1.5 us; 28672 x
// 8192: 94 against 112, and stretches are faster by 5 us).
FewPlan few_plan(int N, int K) {
  FewPlan p{};
  p.blocks = ceil_div(N, FEW_CH);
  p.steps = ceil_div(K, FEW_K);
  const long long units = static_cast<long long>(p.blocks) * p.steps;
  const long long whole = static_cast<long long>(ceil_div(p.blocks, Q8_SMS)) * p.steps, even = units / Q8_SMS + 6;
  p.ctas = static_cast<int>(whole <= even ? p.blocks : std::min<long long>(units, FEW_CTAS * Q8_SMS));
  p.total = p.ctas == p.blocks ? 0 : sizeof(int) * FEW_SLOT * 2 * static_cast<size_t>(p.ctas);
  return p;
}

// Unit u of blocks x steps at which CTA c of `ctas` begins.
__host__ __device__ __forceinline__ long long first_unit(long long units, int ctas, int c) { return units * c / ctas; }

template <int DT>
__device__ __forceinline__ void few_store(const Q8Args& a, int ch, int row, int sum) {
  if (ch >= a.N || row >= a.M) return;
  float v = static_cast<float>(sum) * load_global(a.x_scales + row) * load_global(a.w_scales + ch);
  if (a.bias != nullptr) v += load16<DT>(a.bias, ch);
  static_cast<uint16_t*>(a.out)[static_cast<size_t>(row) * a.N + ch] = static_cast<uint16_t>(pack2<DT>(v, 0.0f));
}

// Up to 8 rows.  A CTA takes a stretch of the steps of all blocks of 16 channels, its
// warps 128 codes of a step each.  A lane's 16 bytes of a weight row and of a token are
// the operands of two instructions (the order of K within them is the lanes' own, the
// same for both sides).  Weights and tokens are loaded FEW_DEPTH steps ahead into
// registers.  The warps' sums meet in shared memory at the end of a block; a block
// that a CTA has only a part of goes to the workspace, two places for each CTA, and
// q8_few_join_kernel adds the parts.
//
// The 8-bit instruction is no faster than 16 cycles an SM, so that 16 rows would be
// bound by it (13 rows of 28672 x 8192: 70 us, tensor pipe 75 % busy).  1 to 8 rows of
// 28672 x 8192: 44 us and the join, 5.4 TB/s, tensor pipe 63 %; of 4096 x 4096: 4.6 us,
// latency.  128 codes of a row together are whole lines: 14336 x 4096 16 us, 64 18.
template <int DT>
__global__ void __launch_bounds__(FEW_THREADS, FEW_CTAS)
q8_few_kernel(const __grid_constant__ Q8Args a, int* parts, int steps, long long units) {
  __shared__ int red[FEW_WARPS][FEW_SLOT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const long long u0 = first_unit(units, gridDim.x, blockIdx.x), u1 = first_unit(units, gridDim.x, blockIdx.x + 1);
  const int first_block = static_cast<int>(u0 / steps), first_step = static_cast<int>(u0 - static_cast<long long>(first_block) * steps);
  int left_a = static_cast<int>(u1 - u0), left = left_a;  // steps to fetch, to work on
  // what is fetched next: 16 bytes of channels g and g + 8 of a block, and of token g
  const size_t pitch = static_cast<size_t>(a.K);
  int step_a = first_step, k_a = first_step * FEW_K + warp * 128 + t * 16, n_a = first_block * FEW_CH + g;
  const int8_t* w_a = a.w + static_cast<size_t>(n_a) * pitch + k_a;
  const int8_t* x_a = a.x + static_cast<size_t>(g) * pitch + k_a;
  wait_for_previous();
  uint4 lo[FEW_DEPTH][2], hi[FEW_DEPTH][2], xs[FEW_DEPTH][2];
  const uint4 none = make_uint4(0, 0, 0, 0);
  auto fetch = [&](uint4 (&l)[2], uint4 (&h)[2], uint4 (&x)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = left_a > 0 && k_a + 64 * j < a.K;
      l[j] = in && n_a < a.N ? load_global(reinterpret_cast<const uint4*>(w_a + 64 * j)) : none;
      h[j] = in && n_a + 8 < a.N ? load_global(reinterpret_cast<const uint4*>(w_a + 8 * pitch + 64 * j)) : none;
      x[j] = in && g < a.M ? load_global(reinterpret_cast<const uint4*>(x_a + 64 * j)) : none;
    }
    --left_a;
    if (++step_a < steps) {
      k_a += FEW_K;
      w_a += FEW_K;
      x_a += FEW_K;
    } else {  // the next block's first step
      const int back = (steps - 1) * FEW_K;
      step_a = 0;
      k_a -= back;
      x_a -= back;
      n_a += FEW_CH;
      w_a += FEW_CH * pitch - back;
    }
  };
#pragma unroll
  for (int i = 0; i < FEW_DEPTH; ++i) fetch(lo[i], hi[i], xs[i]);
  int acc[4] = {};
  int block = first_block, step = first_step;
  bool from_start = step == 0, first = true;
  while (left > 0) {
#pragma unroll
    for (int i = 0; i < FEW_DEPTH; ++i) {
      if (left == 0) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_s8(acc, lo[i][j].x, hi[i][j].x, lo[i][j].y, hi[i][j].y, xs[i][j].x, xs[i][j].y);
        mma_s8(acc, lo[i][j].z, hi[i][j].z, lo[i][j].w, hi[i][j].w, xs[i][j].z, xs[i][j].w);
      }
      fetch(lo[i], hi[i], xs[i]);
      --left;
      const bool ends = ++step == steps;
      if (ends || left == 0) {
        // a lane's sums: channels g and g + 8 of rows 2 t and 2 t + 1
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          red[warp][(2 * t + (c & 1)) * FEW_CH + g + (c & 2) * 4] = acc[c];
          acc[c] = 0;
        }
        __syncthreads();
        if (threadIdx.x < FEW_SLOT) {
          const int o = threadIdx.x;
          int s = 0;
#pragma unroll
          for (int v = 0; v < FEW_WARPS; ++v) s += red[v][o];
          if (ends && from_start) few_store<DT>(a, block * FEW_CH + o % FEW_CH, o / FEW_CH, s);
          else parts[(2 * static_cast<size_t>(blockIdx.x) + (first ? 0 : 1)) * FEW_SLOT + o] = s;
        }
        __syncthreads();
        first = false;
        from_start = true;
        step = 0;
        ++block;
      }
    }
  }
}

// Adds the parts of the block that CTA b - 1 and CTA b share, if b is the first to
// continue it, and leaves them zero.
template <int DT>
__global__ void __launch_bounds__(FEW_SLOT)
q8_few_join_kernel(const __grid_constant__ Q8Args a, int* parts, int steps, long long units, int ctas) {
  wait_for_previous();
  const int b = blockIdx.x + 1, o = threadIdx.x;
  const long long at = first_unit(units, ctas, b);
  const int block = static_cast<int>(at / steps);
  const long long begin = static_cast<long long>(block) * steps, end = begin + steps;
  if (at == begin || first_unit(units, ctas, b - 1) > begin) return;
  int s = 0;
  for (int c = b - 1; c < ctas; ++c) {
    const long long u0 = first_unit(units, ctas, c);
    if (u0 >= end) break;
    // a CTA's first block is in its first place, the one it ends in the second
    int* p = parts + (2 * static_cast<size_t>(c) + (u0 >= begin ? 0 : 1)) * FEW_SLOT + o;
    s += *p;
    *p = 0;
  }
  few_store<DT>(a, block * FEW_CH + o % FEW_CH, o / FEW_CH, s);
}

template <int DT>
flux_status_t few_rows(const Q8Args& a, void* workspace, cudaStream_t s) {
  const FewPlan p = few_plan(a.N, a.K);
  int* parts = reinterpret_cast<int*>(static_cast<char*>(workspace) + WS_HEADER);
  const long long units = static_cast<long long>(p.blocks) * p.steps;
  cudaError_t e = launch_behind(q8_few_kernel<DT>, dim3(p.ctas), FEW_THREADS, 0, s, a, parts, p.steps, units);
  if (e == cudaSuccess && p.ctas != p.blocks)
    e = launch_behind(q8_few_join_kernel<DT>, dim3(p.ctas - 1), FEW_SLOT, 0, s, a, parts, p.steps, units, p.ctas);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

// K = 0: the bias, or zeros.
template <int DT>
__global__ void q8_empty_kernel(const __grid_constant__ Q8Args a) {
  const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<size_t>(a.M) * a.N) return;
  static_cast<uint16_t*>(a.out)[i] = a.bias != nullptr ? static_cast<const uint16_t*>(a.bias)[i % a.N] : 0;
}

template <int DT>
flux_status_t quantize(int rows, int K, const void* x, int8_t* q, float* scales, cudaStream_t s) {
  const int nvec = K / 8;
  cudaError_t e;
  if (nvec <= 128 * QZ_VECS) e = launch_behind(q8_quantize_kernel<DT, 128>, dim3(rows), 128, 0, s, x, q, scales, K);
  else if (nvec <= 512 * QZ_VECS) e = launch_behind(q8_quantize_kernel<DT, 512>, dim3(rows), 512, 0, s, x, q, scales, K);
  else e = launch_behind(q8_quantize_kernel<DT, 1024>, dim3(rows), 1024, 0, s, x, q, scales, K);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

bool q8_sizes_ok(int M, int N, int K) { return M >= 0 && N >= 0 && K >= 0; }
bool q8_sizes_supported(int M, int N, int K) {
  return K % 16 == 0 && K <= Q8_MAX_K && N % 8 == 0 && N <= (1 << 30) && M <= (1 << 30);
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" flux_status_t flux_q8_quantize(int rows, int K, flux_dtype_t dtype, const void* x, int8_t* q, float* scales,
                                          void* stream) {
  if (rows < 0 || K < 0 || (dtype != FLUX_F16 && dtype != FLUX_BF16)) return FLUX_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > Q8_MAX_K) return FLUX_ERR_UNSUPPORTED;
  if (rows == 0) return FLUX_OK;
  if (scales == nullptr || (K > 0 && (x == nullptr || q == nullptr))) return FLUX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales)) return FLUX_ERR_UNSUPPORTED;
  DeviceInfo dev;
  flux_status_t st = current_device(&dev);
  if (st != FLUX_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == FLUX_BF16 ? quantize<1>(rows, K, x, q, scales, s) : quantize<0>(rows, K, x, q, scales, s);
}

extern "C" size_t flux_q8_workspace_size(int M, int N, int K) {
  if (!q8_sizes_ok(M, N, K) || !q8_sizes_supported(M, N, K)) return 0;
  if (M == 0 || N == 0 || K == 0) return WS_HEADER;
  const size_t few = few_plan(N, K).total;
  return WS_HEADER + (M <= FEW_ROWS ? few : std::max(few, q8_gemm_most_bytes(M, N, K)));
}

extern "C" flux_status_t flux_q8_gemm(int M, int N, int K, flux_dtype_t dtype, const int8_t* x, const float* x_scales,
                                      const int8_t* w, const float* w_scales, const void* bias, void* out,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!q8_sizes_ok(M, N, K) || (dtype != FLUX_F16 && dtype != FLUX_BF16)) return FLUX_ERR_INVALID_ARG;
  if (!q8_sizes_supported(M, N, K)) return FLUX_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return FLUX_OK;
  if (out == nullptr || (K > 0 && (x == nullptr || w == nullptr || x_scales == nullptr || w_scales == nullptr)))
    return FLUX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(x_scales) || !aligned16(w_scales) || !aligned16(bias) || !aligned16(out))
    return FLUX_ERR_UNSUPPORTED;
  const size_t need = K == 0 ? 0 : M <= FEW_ROWS ? few_plan(N, K).total : q8_gemm_bytes(M, N, K);
  flux_status_t st = check_workspace(workspace, workspace_bytes, WS_HEADER + need);
  if (st != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Q8Args a{x, x_scales, w, w_scales, bias, out, M, N, K};
  if (K == 0) {
    const size_t n = static_cast<size_t>(M) * N;
    q8_empty_kernel<0><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  }
  if (M <= FEW_ROWS) return dtype == FLUX_BF16 ? few_rows<1>(a, workspace, s) : few_rows<0>(a, workspace, s);
  return q8_gemm_launch(a, dtype, workspace, dev, s);
}
