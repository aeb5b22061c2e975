// 8-bit products of many rows.  The codes are widened to fp16, which holds them
// exactly, and multiplied by tcgen05.mma kind::f16: the products are exact, and so
// are the fp32 sums while they stay below 2^24 (always up to K = 1040; with codes of
// ordinary spread at every K), beyond that each step of 16 rounds to 24 bits.
//
// A pair of CTAs computes 256 rows x 256 channels at a time (128 rows and 128 of
// the channels' codes in each CTA's shared memory, 6 stages of 64 codes); two
// accumulators of 256 columns, so that the scaling and storing of one tile runs
// under the matrix products of the next.
#include <algorithm>

#include "flux_kernels.cuh"
#include "flux_q8.h"

namespace flux {

namespace {

constexpr int G_BK = 64, G_STAGES = 6, G_TILE = 256, G_ROWS = 128;  // rows of either operand in one CTA
constexpr int G_OPERAND = G_ROWS * G_BK * 2, G_STAGE = 2 * G_OPERAND;
constexpr int G_SMEM = G_STAGES * G_STAGE + 1024 + 256;
constexpr int G_THREADS = 6 * 32;  // a warp that loads, one that multiplies, four that store
constexpr int G_BAND = 8;          // row tiles that are worked through together

struct Q8GemmParams {
  CUtensorMap x, w;  // widened codes [rows x K]
  Q8Args a;
  uint32_t* hdr;
  uint32_t seq;
  uint64_t timeout_ns;
  int Mt, Nt, KT;
};

// 16 codes to fp16: 1024 + (code + 128) is the number whose low mantissa bits are
// the biased byte.
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi) {
  v ^= 0x80808080u;
  const uint32_t a = __byte_perm(v, 0x64646464u, 0x4140), b = __byte_perm(v, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), bias), hb = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&ha);
  hi = *reinterpret_cast<const uint32_t*>(&hb);
}

__global__ void __launch_bounds__(256)
q8_widen_kernel(const uint4* __restrict__ x, uint4* __restrict__ xf, size_t nx, const uint4* __restrict__ w,
                uint4* __restrict__ wf, size_t nw) {
  const size_t step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < nx + nw; i += step) {
    const bool is_x = i < nx;
    const size_t at = is_x ? i : i - nx;
    const uint4 v = __ldg((is_x ? x : w) + at);
    uint4 o[2];
    widen(v.x, o[0].x, o[0].y);
    widen(v.y, o[0].z, o[0].w);
    widen(v.z, o[1].x, o[1].y);
    widen(v.w, o[1].z, o[1].w);
    uint4* dst = (is_x ? xf : wf) + 2 * at;
    dst[0] = o[0];
    dst[1] = o[1];
  }
}

// Tile t: bands of G_BAND row tiles, in a band column by column.
__device__ __forceinline__ void tile_at(const Q8GemmParams& p, int t, int& mt, int& nt) {
  const int per = G_BAND * p.Nt, band = t / per, rest = t - band * per;
  const int rows = min(G_BAND, p.Mt - band * G_BAND);
  nt = rest / rows;
  mt = band * G_BAND + rest - nt * rows;
}

template <int DT>
__global__ void __launch_bounds__(G_THREADS, 1)
q8_gemm_kernel(const __grid_constant__ Q8GemmParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + G_STAGES * G_STAGE);
  uint64_t *full = bars, *empty = bars + G_STAGES, *tfull = empty + G_STAGES, *tempty = tfull + 2, *drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const Ctl c{p.hdr, p.seq, p.timeout_ns, 2 * p.timeout_ns + 10000000ull};
  if (threadIdx.x == 0) {
    for (int i = 0; i < G_STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 8);  // four warps of either CTA
    }
    mbar_init(smem_u32(drain), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2, tiles = p.Mt * p.Nt;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&p.x);
      tma_prefetch_desc(&p.w);
      uint32_t stage = 0, phase = 0, issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs) {
        int mt, nt;
        tile_at(p, t, mt, nt);
        const int row = mt * G_TILE + static_cast<int>(cta) * G_ROWS, ch = nt * G_TILE + static_cast<int>(cta) * G_ROWS;
        for (int k = 0; k < p.KT; ++k) {
          if (wait_bar(smem_u32(&empty[stage]), phase ^ 1u, c, W_EMPTY, stage) != 0) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[stage]);
          // the even CTA's barrier counts both CTAs' bytes
          if (cta == 0) mbar_arrive_expect_tx(fb, 2 * G_STAGE);
          const uint32_t fbc = mapa_shared(fb, 0u), dst = smem_u32(base + stage * G_STAGE);
          tma_load_2d_pair(dst, &p.x, fbc, k * G_BK, row);
          tma_load_2d_pair(dst + G_OPERAND, &p.w, fbc, k * G_BK, ch);
          ++issued;
          if (++stage == G_STAGES) stage = 0, phase ^= 1u;
        }
      }
      // every issued copy lands before the CTA may exit; the odd CTA sees its own
      // only by the products that read them
      for (uint32_t st = 0; st < G_STAGES; ++st) {
        const uint32_t fills = issued / G_STAGES + (st < issued % G_STAGES ? 1u : 0u);
        if (fills == 0) continue;
        if (cta != 0) wait_bar_remote_drain(smem_u32(&empty[st]), (fills - 1u) & 1u, c, W_DRAIN, st);
        else wait_bar(smem_u32(&full[st]), (fills - 1u) & 1u, c, W_DRAIN, st, false);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && cta == 0) {
      constexpr uint32_t IDESC = idesc_f16(0, 256, 256, 0, 0);
      uint32_t stage = 0, phase = 0;
      int it = 0;
      bool ok = true, any = false;
      for (int t = pair; ok && t < tiles; t += pairs, ++it) {
        const uint32_t b = it & 1, use = static_cast<uint32_t>(it >> 1);
        const uint32_t d = tmem + b * 256;
        if (wait_bar_remote(smem_u32(&tempty[b]), (use & 1u) ^ 1u, c, W_TEMPTY, b) != 0) break;
        tc_fence_after();
        for (int k = 0; k < p.KT; ++k) {
          if (wait_bar(smem_u32(&full[stage]), phase, c, W_FULL, stage) != 0) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(base + stage * G_STAGE);
#pragma unroll
          for (int kk = 0; kk < G_BK / 16; ++kk) {
            // both K-major: rows of 128 bytes, groups of 8 rows 1024 bytes apart, 16 codes 32 bytes
            const uint64_t ad = sdesc_sw128(sa + kk * 32, 16, 1024), bd = sdesc_sw128(sa + G_OPERAND + kk * 32, 16, 1024);
            umma2_f16(d, ad, bd, IDESC, (k > 0 || kk > 0) ? 1u : 0u);
          }
          umma2_commit_mc(smem_u32(&empty[stage]), 3);
          any = true;
          if (++stage == G_STAGES) stage = 0, phase ^= 1u;
        }
        if (ok) umma2_commit_mc(smem_u32(&tfull[b]), 3);
      }
      if (any) {
        umma2_commit(smem_u32(drain));
        wait_bar(smem_u32(drain), 0, c, W_DRAIN, 0, false);
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    int it = 0;
    for (int t = pair; t < tiles; t += pairs, ++it) {
      int mt, nt;
      tile_at(p, t, mt, nt);
      const uint32_t b = it & 1, use = static_cast<uint32_t>(it >> 1);
      if (wait_bar_remote(smem_u32(&tfull[b]), use & 1u, c, W_TFULL, b) != 0) break;
      __syncwarp();
      tc_fence_after();
      const int row = mt * G_TILE + static_cast<int>(cta) * G_ROWS + quarter * 32 + lane;
      const bool in = row < p.a.M;
      const float xs = in ? __ldg(p.a.x_scales + row) : 0.0f;
      uint16_t* dst = static_cast<uint16_t*>(p.a.out) + static_cast<size_t>(row) * p.a.N;
      for (int c0 = 0; c0 < G_TILE; c0 += 32) {
        const int ch0 = nt * G_TILE + c0;
        if (ch0 >= p.a.N) break;
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + b * 256 + c0 + (static_cast<uint32_t>(quarter) * 32u << 16), r);
        const float ws = ch0 + lane < p.a.N ? __ldg(p.a.w_scales + ch0 + lane) : 0.0f;
        float bias = 0.0f;
        if (p.a.bias != nullptr && ch0 + lane < p.a.N) {
          const uint16_t h = __ldg(static_cast<const uint16_t*>(p.a.bias) + ch0 + lane);
          bias = DT == 1 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float s = __shfl_sync(0xFFFFFFFFu, ws, j), o = __shfl_sync(0xFFFFFFFFu, bias, j);
          r[j] = __float_as_uint(__uint_as_float(r[j]) * xs * s + o);
        }
        if (in) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (ch0 + j < p.a.N) {
              auto two = [&](int i) { return pack2<DT>(__uint_as_float(r[j + i]), __uint_as_float(r[j + i + 1])); };
              *reinterpret_cast<uint4*>(dst + ch0 + j) = make_uint4(two(0), two(2), two(4), two(6));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[b]), 0u));
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

size_t operand_bytes(int rows, int K) {
  return round_up(static_cast<size_t>(ceil_div(rows, G_ROWS)) * G_ROWS * K * 2, WS_ALIGN);
}

template <int DT>
flux_status_t launch(const Q8GemmParams& p, const DeviceInfo& dev, cudaStream_t s) {
  constexpr auto kernel = q8_gemm_kernel<DT>;
  static OncePerDevice once;
  const cudaError_t attr = once(dev.device, [] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM); });
  if (attr != cudaSuccess) return cuda_fail(attr);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::min<long long>(dev.sm_count / 2, static_cast<long long>(p.Mt) * p.Nt), 1, 1);
  cfg.blockDim = dim3(G_THREADS, 1, 1);
  cfg.dynamicSmemBytes = G_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

}  // namespace

size_t q8_gemm_bytes(int M, int N, int K) { return operand_bytes(M, K) + operand_bytes(N, K); }

flux_status_t q8_gemm_launch(const Q8Args& a, flux_dtype_t dtype, void* workspace, const DeviceInfo& dev, cudaStream_t s) {
  char* at = static_cast<char*>(workspace) + WS_HEADER;
  void *xf = at, *wf = at + operand_bytes(a.M, a.K);
  const size_t nx = static_cast<size_t>(a.M) * a.K / 16, nw = static_cast<size_t>(a.N) * a.K / 16;
  const size_t blocks = std::min<size_t>((nx + nw + 255) / 256, static_cast<size_t>(dev.sm_count) * 8);
  q8_widen_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(
      reinterpret_cast<const uint4*>(a.x), static_cast<uint4*>(xf), nx, reinterpret_cast<const uint4*>(a.w), static_cast<uint4*>(wf), nw);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  Q8GemmParams p{};
  // whole blocks of rows: what lies past the last row is read, and never stored
  flux_status_t st = encode_2d(&p.x, FLUX_F16, xf, a.K, static_cast<uint64_t>(ceil_div(a.M, G_ROWS)) * G_ROWS, a.K * 2ull, G_BK, G_ROWS);
  if (st == FLUX_OK)
    st = encode_2d(&p.w, FLUX_F16, wf, a.K, static_cast<uint64_t>(ceil_div(a.N, G_ROWS)) * G_ROWS, a.K * 2ull, G_BK, G_ROWS);
  if (st != FLUX_OK) return st;
  p.a = a;
  p.hdr = static_cast<uint32_t*>(workspace);
  p.seq = next_seq();
  p.timeout_ns = DEFAULT_TIMEOUT_NS;
  p.Mt = ceil_div(a.M, G_TILE);
  p.Nt = ceil_div(a.N, G_TILE);
  p.KT = ceil_div(a.K, G_BK);
  return dtype == FLUX_BF16 ? launch<1>(p, dev, s) : launch<0>(p, dev, s);
}

}  // namespace flux
