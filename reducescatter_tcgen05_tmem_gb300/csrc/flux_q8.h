// 8-bit products: what the entry point (flux_q8.cu) and the tensor-core GEMM
// (flux_q8_gemm.cu) share.
#pragma once

#include "flux_host.h"

namespace flux {

struct Q8Args {
  const int8_t* x;       // [M x K]
  const float* x_scales; // [M]
  const int8_t* w;       // [N x K]
  const float* w_scales; // [N]
  const void* bias;      // [N] or null
  void* out;             // [M x N]
  int M, N, K;
};

// The GEMM of many rows: its workspace (past the header) for this size, and for every
// M up to this; its launch.
size_t q8_gemm_bytes(int M, int N, int K);
size_t q8_gemm_most_bytes(int M, int N, int K);
flux_status_t q8_gemm_launch(const Q8Args& a, flux_dtype_t dtype, void* workspace, const DeviceInfo& dev,
                             cudaStream_t s);

}  // namespace flux
