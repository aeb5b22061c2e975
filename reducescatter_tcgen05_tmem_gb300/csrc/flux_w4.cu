// Products of few rows with 4-bit weights: out = x . W, W[k, n] = scale[k / group, n] (code[n, k] - 8).
//
// With a handful of rows such a product does 2 M operations per half byte of
// weights, so it is bound by reading the weights once.  They are stored
// column by column, 128 inputs (64 bytes) at a time, in the order in which
// the lanes of a warp use them: in each run of 128 inputs, 16 bytes for every
// c of 0..3, in them one 32-bit word for every j of 0..3, whose nibbles i and
// i + 4 hold the inputs 32 j + 8 c + 2 i and 32 j + 8 c + 2 i + 1.
#include <math.h>

#include <algorithm>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int W4_RUN = 128;  // inputs per run of 64 bytes

enum W4Mode { W4_DENSE = 0, W4_LAYER0 = 1, W4_LAYER1 = 2 };

struct W4Args {
  const void* x;
  const uint8_t* q;
  const void* scales;
  const int32_t* ids;
  const float* weights;
  void* out;
  uint32_t* hdr;
  int rows;  // output rows: M, T topk (layer0), T (layer1)
  int N, K, runs, group, groups, E, topk, mode;
};

// One warp per output column and row.
template <int DT>
__global__ void __launch_bounds__(256) w4_kernel(const __grid_constant__ W4Args a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x * 8 + warp;
  if (n >= a.N) return;
  for (int r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const int slots = a.mode == W4_LAYER1 ? a.topk : 1;
    float total = 0.0f;
    for (int j = 0; j < slots; ++j) {
      const int slot = a.mode == W4_LAYER1 ? r * a.topk + j : r;
      int e = 0;
      if (a.mode != W4_DENSE) {
        e = a.ids[slot];
        if (e < 0 || e >= a.E) {
          if (lane == 0 && n == 0) atomicCAS(a.hdr, 0u, static_cast<uint32_t>(FLUX_ERR_INVALID_ARG));
          continue;
        }
      }
      const size_t xrow = static_cast<size_t>(a.mode == W4_LAYER0 ? r / a.topk : slot) * a.K;
      const uint32_t* q =
          reinterpret_cast<const uint32_t*>(a.q + (static_cast<size_t>(e) * a.N + n) * a.runs * (W4_RUN / 2));
      float sum = 0.0f;
      for (int w = lane; w < a.runs * 16; w += 32) {
        const int k0 = w / 16 * W4_RUN + w % 4 * 32 + w / 4 % 4 * 8;
        if (k0 >= a.K) continue;
        const uint32_t v = q[w];
        const float scale = load16<DT>(a.scales, (static_cast<size_t>(e) * a.groups + k0 / a.group) * a.N + n);
        float xs[8], part = 0.0f;
        unpack8<DT>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + xrow + k0)), xs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          part += xs[2 * i] * static_cast<float>(static_cast<int>(v >> (4 * i) & 15u) - 8);
          part += xs[2 * i + 1] * static_cast<float>(static_cast<int>(v >> (4 * i + 16) & 15u) - 8);
        }
        sum += part * scale;
      }
      sum = warp_sum(sum);
      total += a.mode == W4_LAYER1 ? a.weights[slot] * sum : sum;
    }
    if (lane == 0)
      static_cast<uint16_t*>(a.out)[static_cast<size_t>(r) * a.N + n] = static_cast<uint16_t>(pack2<DT>(total, 0.0f));
  }
}

// One thread per column and group: the group's largest magnitude / 7, rounded
// to 16 bits, is its scale; codes are the nearest multiples of it.
template <int DT>
__global__ void __launch_bounds__(128)
w4_quantize_kernel(int K, int N, int runs, int group, int groups, const void* __restrict__ w, uint8_t* __restrict__ q,
                   void* __restrict__ scales) {
  const int n = blockIdx.x * 128 + threadIdx.x;
  const size_t e = blockIdx.z;
  if (n >= N) return;
  const size_t wbase = e * K * N + n;
  for (int g = blockIdx.y; g < groups; g += gridDim.y) {
    const int k0 = g * group, k1 = min(k0 + group, K);
    float top = 0.0f;
    for (int k = k0; k < k1; ++k) top = fmaxf(top, fabsf(load16<DT>(w, wbase + static_cast<size_t>(k) * N)));
    const uint32_t s16 = pack2<DT>(top / 7.0f, 0.0f);
    const float scale = unpack2<DT>(s16).x;
    static_cast<uint16_t*>(scales)[(e * groups + g) * N + n] = static_cast<uint16_t>(s16);
    // the last group also fills its run of 128 inputs
    const int kend = g == groups - 1 ? runs * W4_RUN : k1;
    for (int k = k0; k < kend; k += 8) {
      uint32_t word = 0x88888888u;
      if (k < K && scale > 0.0f) {
        word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = load16<DT>(w, wbase + static_cast<size_t>(k + i) * N);
          const int code = min(max(static_cast<int>(rintf(v / scale)) + 8, 0), 15);
          word |= static_cast<uint32_t>(code) << (i / 2 * 4 + i % 2 * 16);
        }
      }
      const int r = k % W4_RUN;
      *reinterpret_cast<uint32_t*>(q + ((e * N + n) * runs + k / W4_RUN) * (W4_RUN / 2) + r % 32 / 8 * 16 + r / 32 * 4) =
          word;
    }
  }
}

bool w4_common_ok(int N, int K, int group, int E, flux_dtype_t dtype) {
  return N >= 0 && K >= 0 && group >= 1 && E >= 1 && E <= FLUX_MAX_EXPERTS && (dtype == FLUX_F16 || dtype == FLUX_BF16);
}

flux_status_t w4_run(W4Mode mode, int rows, int xrows, int T, int N, int K, int E, int topk, int group,
                     flux_dtype_t dtype, const void* x, const void* q, const void* scales, const int32_t* ids,
                     const float* weights, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || !w4_common_ok(N, K, group, E, dtype) || topk < 1 || topk > E) return FLUX_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0 || group % 32 != 0) return FLUX_ERR_UNSUPPORTED;
  if (static_cast<long long>(T) * topk > FLUX_W4_MAX_ROWS) return FLUX_ERR_UNSUPPORTED;
  if (rows == 0 || N == 0) return FLUX_OK;
  if (out == nullptr || (K > 0 && (x == nullptr || q == nullptr || scales == nullptr)) ||
      (mode != W4_DENSE && ids == nullptr) || (mode == W4_LAYER1 && weights == nullptr))
    return FLUX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || !aligned16(ids) || !aligned16(weights) || !aligned16(out))
    return FLUX_ERR_UNSUPPORTED;
  flux_status_t st = check_workspace(workspace, workspace_bytes, flux_w4_workspace_size(xrows, N, K, E));
  if (st != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  W4Args a{};
  a.x = x;
  a.q = static_cast<const uint8_t*>(q);
  a.scales = scales;
  a.ids = ids;
  a.weights = weights;
  a.out = out;
  a.hdr = static_cast<uint32_t*>(workspace);
  a.rows = rows;
  a.N = N;
  a.K = K;
  a.runs = (K + W4_RUN - 1) / W4_RUN;
  a.group = group;
  a.groups = (K + group - 1) / group;
  a.E = E;
  a.topk = topk;
  a.mode = mode;
  const dim3 grid((N + 7) / 8, rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FLUX_BF16) w4_kernel<1><<<grid, 256, 0, s>>>(a);
  else w4_kernel<0><<<grid, 256, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" size_t flux_w4_weight_bytes(int E, int K, int N) {
  if (E < 1 || K < 0 || N < 0) return 0;
  return static_cast<size_t>(E) * N * ((K + W4_RUN - 1) / W4_RUN) * (W4_RUN / 2);
}

extern "C" size_t flux_w4_workspace_size(int rows, int N, int K, int E) {
  if (rows < 0 || rows > FLUX_W4_MAX_ROWS || N < 0 || K < 0 || E < 1 || E > FLUX_MAX_EXPERTS) return 0;
  return WS_HEADER;
}

extern "C" flux_status_t flux_w4_quantize(int E, int K, int N, int group, flux_dtype_t dtype, const void* w, void* q,
                                          void* scales, void* stream) {
  if (!w4_common_ok(N, K, group, E, dtype)) return FLUX_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0 || group % 32 != 0) return FLUX_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return FLUX_OK;
  if (w == nullptr || q == nullptr || scales == nullptr) return FLUX_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(q) || !aligned16(scales)) return FLUX_ERR_UNSUPPORTED;
  DeviceInfo dev;
  flux_status_t st = current_device(&dev);
  if (st != FLUX_OK) return st;
  const int runs = (K + W4_RUN - 1) / W4_RUN, groups = (K + group - 1) / group;
  const dim3 grid((N + 127) / 128, std::min(groups, 65535), E);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FLUX_BF16)
    w4_quantize_kernel<1><<<grid, 128, 0, s>>>(K, N, runs, group, groups, w, static_cast<uint8_t*>(q), scales);
  else
    w4_quantize_kernel<0><<<grid, 128, 0, s>>>(K, N, runs, group, groups, w, static_cast<uint8_t*>(q), scales);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

extern "C" flux_status_t flux_w4_gemv(int M, int N, int K, int group, flux_dtype_t dtype, const void* x, const void* q,
                                      const void* scales, void* out, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  return w4_run(W4_DENSE, M, M, M, N, K, 1, 1, group, dtype, x, q, scales, nullptr, nullptr, out, workspace,
                workspace_bytes, stream);
}

extern "C" flux_status_t flux_moe_w4_layer0(int T, int H, int F, int E, int topk, int group, flux_dtype_t dtype,
                                            const void* x, const void* q1, const void* scales1,
                                            const int32_t* topk_ids, void* h, void* workspace, size_t workspace_bytes,
                                            void* stream) {
  const long long slots = static_cast<long long>(T) * topk;
  const int n = slots < 0 || slots > FLUX_W4_MAX_ROWS ? 0 : static_cast<int>(slots);
  return w4_run(W4_LAYER0, n, n, T, F, H, E, topk, group, dtype, x, q1, scales1, topk_ids, nullptr, h, workspace,
                workspace_bytes, stream);
}

extern "C" flux_status_t flux_moe_w4_layer1(int T, int H, int F, int E, int topk, int group, flux_dtype_t dtype,
                                            const void* h, const void* q2, const void* scales2,
                                            const int32_t* topk_ids, const float* topk_weights, void* out,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  const long long slots = static_cast<long long>(T) * topk;
  const int n = slots < 0 || slots > FLUX_W4_MAX_ROWS ? 0 : static_cast<int>(slots);
  return w4_run(W4_LAYER1, T, n, T, H, F, E, topk, group, dtype, h, q2, scales2, topk_ids, topk_weights, out,
                workspace, workspace_bytes, stream);
}
