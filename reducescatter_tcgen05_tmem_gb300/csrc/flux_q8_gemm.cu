// 8-bit products of more than a few rows, on the 16-bit tensor cores: fp16 holds the
// codes and their products exactly, and so does the fp32 sum while it stays below
// 2^24 (always up to K = 1024; with codes of ordinary spread at every K), beyond that
// each step of 16 rounds to 24 bits, so that the error grows with K (large codes of one
// sign: 4e-5 of the sum at K = 131056).
//
// out^T = w x^T: the channels are the rows of the tensor core's product and the tokens
// its columns, of which there may be any multiple of 16, so that few tokens cost
// little.  The weights travel as they are held, in bytes: TMA brings them into shared
// memory, eight warps widen them and put them into TMEM, where tcgen05.mma takes its
// left operand from.  In shared memory the widened weights would be written and read
// again, which its 128 bytes a cycle cannot feed beside the products (staged that way
// 4096 x 4096 x 14336 took 323 us).  The tokens, which every channel tile reads, are
// widened once by a small kernel before.
//
// A pair of CTAs computes 256 channels x up to 160 tokens (tcgen05.mma.cta_group::2,
// 128 channels and half of the tokens' codes in each CTA).  TMEM: two accumulators of
// 160 columns, so that one tile is scaled and stored under the products of the next,
// and three buffers of the widened codes of a step (with 192 columns there is room for
// two, and a buffer's round, products, commit, widening, arrival, takes longer than the
// products of the other: 4096 x 4096 x 14336 320 us).  Where there are fewer tiles than
// pairs K is cut into parts, whose fp32 sums q8_parts_kernel adds in order.
//
// 4096 tokens, 14336 channels of 4096: this kernel 246 us, 1.95 PFLOP/s, tensor pipe 90 %
// busy.  333 tokens, 4096 channels of 14336: 36 us, 53 % (K in three parts, whose 16 MB of
// sums the next kernel adds in 8).  13 tokens, 8192 channels of 28672: 47 us, 5 TB/s.
#include <limits.h>

#include <algorithm>

#include "flux_kernels.cuh"
#include "flux_q8.h"

namespace flux {

namespace {

constexpr int G_K = 128;                 // codes of a step
constexpr int G_CH = 256, G_ROWS = 128;  // channels of a tile, of a CTA
constexpr int G_TOK = 160;               // most tokens of a tile
constexpr int G_RAW = G_ROWS * G_K, G_RAW_STAGES = 6;
constexpr int G_ATOM = G_TOK / 2 * 128;  // 64 widened codes of a CTA's tokens
constexpr int G_TOK_BYTES = 2 * G_ATOM, G_TOK_STAGES = 5;
constexpr int G_A = 2 * G_TOK, G_A_COLS = 64, G_A_BUFS = 3;  // TMEM columns of the widened weights of a step
constexpr int G_SMEM = G_RAW_STAGES * G_RAW + G_TOK_STAGES * G_TOK_BYTES + 1024 + 512;
// warps: 0 weights, 1 tokens, 2 products, 4..7 epilogue, 8..15 widening
constexpr int G_THREADS = 16 * 32;
constexpr int G_BAND = 8;    // channel tiles that are worked through together
constexpr int G_PAIRS = 76;  // pairs at work
static_assert(G_A + G_A_BUFS * G_A_COLS == 512, "TMEM columns");

struct Q8GemmParams {
  CUtensorMap x, w;  // widened tokens [rows x K]; codes [N x K]
  Q8Args a;
  float* parts;      // [splits][M][N], or null where K is not cut
  uint32_t* hdr;
  uint32_t seq;
  uint64_t timeout_ns;
  int n, ch_tiles, tok_tiles, steps, splits;
};

// (as in flux_rows.cuh, whose pack2 the GEMM headers define too)
template <typename T>
__device__ __forceinline__ T load_global(const T* p) {
  return *p;
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, size_t smem, int cluster, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Four codes to fp16: 1024 + (code + 128) is the number whose low mantissa bits are
// the biased byte.
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi) {
  v ^= 0x80808080u;
  const uint32_t a = __byte_perm(v, 0x64646464u, 0x4140), b = __byte_perm(v, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), bias), hb = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&ha);
  hi = *reinterpret_cast<const uint32_t*>(&hb);
}

__global__ void __launch_bounds__(256) q8_widen_kernel(const uint4* x, uint4* xf, size_t n) {
  after_previous();
  const size_t step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
    const uint4 v = load_global(x + i);
    uint4 o[2];
    widen(v.x, o[0].x, o[0].y);
    widen(v.y, o[0].z, o[0].w);
    widen(v.z, o[1].x, o[1].y);
    widen(v.w, o[1].z, o[1].w);
    xf[2 * i] = o[0];
    xf[2 * i + 1] = o[1];
  }
}

// Unit u: a tile (bands of G_BAND channel tiles, in a band one token tile after the
// other) and a part of its steps.
struct Q8Unit {
  int ct, tt, split, k0, k1;
  __device__ __forceinline__ Q8Unit(const Q8GemmParams& p, int u) {
    const int t = u / p.splits;
    split = u - t * p.splits;
    const int per = G_BAND * p.tok_tiles, band = t / per, rest = t - band * per;
    const int wide = min(G_BAND, p.ch_tiles - band * G_BAND);
    tt = rest / wide;
    ct = band * G_BAND + rest - tt * wide;
    k0 = static_cast<int>(static_cast<long long>(p.steps) * split / p.splits);
    k1 = static_cast<int>(static_cast<long long>(p.steps) * (split + 1) / p.splits);
  }
};

// A converged warp waits.  The first look is inline: a call to the bounded loops costs
// 300 cycles, which a step does not have to spare.  `remote`: the barrier is completed
// by the other CTA too.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Ctl& c, uint32_t where, uint32_t arg, bool remote) {
  if (__all_sync(0xFFFFFFFFu, remote ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) return true;
  const int bad = remote ? wait_bar_remote(bar, parity, c, where, arg) : wait_bar(bar, parity, c, where, arg);
  return !__any_sync(0xFFFFFFFFu, bad != 0);
}

template <int DT>
__global__ void __launch_bounds__(G_THREADS, 1)
q8_gemm_kernel(const __grid_constant__ Q8GemmParams p) {
  extern __shared__ uint8_t smem_base[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_base) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* tok = base + G_RAW_STAGES * G_RAW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(tok + G_TOK_STAGES * G_TOK_BYTES);
  uint64_t *rawfull = bars, *rawempty = rawfull + G_RAW_STAGES, *full = rawempty + G_RAW_STAGES, *done = full + G_TOK_STAGES;
  uint64_t *tfull = done + G_TOK_STAGES, *tempty = tfull + 2, *drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  // (shuffled, so that the compiler knows them to be the same for a warp)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const Ctl c{p.hdr, p.seq, p.timeout_ns, 2 * p.timeout_ns + 10000000ull};
  if (threadIdx.x == 0) {
    for (int i = 0; i < G_RAW_STAGES; ++i) {
      mbar_init(smem_u32(&rawfull[i]), 1);
      mbar_init(smem_u32(&rawempty[i]), 4);  // the widening warps of the step
    }
    for (int i = 0; i < G_TOK_STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 9);  // a step's tokens, and its widening warps of both CTAs
      mbar_init(smem_u32(&done[i]), 1);   // its products
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 8);  // four epilogue warps of either CTA
    }
    mbar_init(smem_u32(drain), 1);
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc2(smem_u32(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
  const int units = p.ch_tiles * p.tok_tiles * p.splits;
  after_previous();

  if (warp == 0) {
    // the weights, into this CTA alone
    if (lane == 0) {
      tma_prefetch_desc(&p.w);
      uint32_t n = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += pairs) {
        const Q8Unit w(p, u);
        const int ch = w.ct * G_CH + static_cast<int>(cta) * G_ROWS;
        for (int k = w.k0; k < w.k1; ++k, ++n) {
          const uint32_t s = n % G_RAW_STAGES;
          if (wait_bar(smem_u32(&rawempty[s]), (n / G_RAW_STAGES & 1u) ^ 1u, c, W_EMPTY, s) != 0) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(smem_u32(&rawfull[s]), G_RAW);
          tma_load_2d(smem_u32(base + s * G_RAW), &p.w, smem_u32(&rawfull[s]), k * G_K, ch);
        }
      }
      // every copy lands before the CTA may exit
      for (uint32_t s = 0; s < G_RAW_STAGES; ++s) {
        const uint32_t fills = n / G_RAW_STAGES + (s < n % G_RAW_STAGES ? 1u : 0u);
        if (fills > 0) wait_bar(smem_u32(&rawfull[s]), (fills - 1u) & 1u, c, W_DRAIN, s, false);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // the tokens; the even CTA's barrier counts both CTAs' bytes
    if (lane == 0) {
      tma_prefetch_desc(&p.x);
      uint32_t n = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += pairs) {
        const Q8Unit w(p, u);
        const int row = w.tt * p.n + static_cast<int>(cta) * (p.n / 2);
        for (int k = w.k0; k < w.k1; ++k, ++n) {
          const uint32_t s = n % G_TOK_STAGES;
          if (wait_bar(smem_u32(&done[s]), (n / G_TOK_STAGES & 1u) ^ 1u, c, W_EMPTY, 16 + s) != 0) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(tok + s * G_TOK_BYTES);
          if (cta == 0) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(p.n) * 256u);
          const uint32_t fbc = mapa_shared(fb, 0u);
          tma_load_2d_pair(dst, &p.x, fbc, k * G_K, row);
          tma_load_2d_pair(dst + G_ATOM, &p.x, fbc, k * G_K + 64, row);
        }
      }
      // the copies have landed when the products that read them are done
      for (uint32_t s = 0; s < G_TOK_STAGES; ++s) {
        const uint32_t fills = n / G_TOK_STAGES + (s < n % G_TOK_STAGES ? 1u : 0u);
        if (fills == 0) continue;
        wait_bar_remote_drain(smem_u32(&done[s]), (fills - 1u) & 1u, c, W_DRAIN, 16 + s);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // The whole warp goes round, one lane issues: an instruction then takes 45 cycles, from
    // a lone thread 90.
    if (cta == 0) {
      const uint32_t idesc = idesc_f16(0, G_CH, p.n, 0, 0);
      uint32_t n = 0;
      int it = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += pairs, ++it) {
        const Q8Unit w(p, u);
        const uint32_t b = it & 1, d = tmem + b * G_TOK;
        ok = warp_wait(smem_u32(&tempty[b]), (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, c, W_TEMPTY, b, true);
        tc_fence_after();
        for (int k = w.k0; ok && k < w.k1; ++k) {
          const uint32_t s = n % G_TOK_STAGES, sb = smem_u32(tok + s * G_TOK_BYTES), ta = tmem + G_A + n % G_A_BUFS * G_A_COLS;
          ok = warp_wait(smem_u32(&full[s]), n / G_TOK_STAGES & 1u, c, W_FULL, 16 + s, true);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              // tokens K-major: rows of 128 bytes, groups of 8 rows 1024 bytes apart
              const uint64_t bd = sdesc_sw128(sb + (kk >> 2) * G_ATOM + (kk & 3) * 32, 16, 1024);
              umma2_f16_tmem_a(d, ta + kk * 8, bd, idesc, (k > w.k0 || kk > 0) ? 1u : 0u);
            }
            umma2_commit_mc(smem_u32(&done[s]), 3);
            if (k + 1 == w.k1) umma2_commit_mc(smem_u32(&tfull[b]), 3);
          }
          __syncwarp();
          ++n;
        }
      }
      if (n > 0) {
        if (elect_one()) umma2_commit(smem_u32(drain));
        if (lane == 0) wait_bar(smem_u32(drain), 0, c, W_DRAIN, 0, false);
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // Widening.  A thread takes the 128 codes of one channel; warps 8..11 the even steps,
    // 12..15 the odd ones, so that a warp waits once for two steps.
    const uint32_t odd = (warp - 8) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = quarter * 32 << 16, raw = smem_u32(base) + row * 128;
    uint32_t n = 0;
    bool ok = true;
    for (int u = pair; ok && u < units; u += pairs) {
      const Q8Unit w(p, u);
      for (int k = w.k0; k < w.k1; ++k, ++n) {
        if ((n & 1u) != odd) continue;
        const uint32_t s = n % G_RAW_STAGES;
        if (!warp_wait(smem_u32(&rawfull[s]), n / G_RAW_STAGES & 1u, c, W_FULL, s, false)) {
          ok = false;
          break;
        }
        const uint32_t src = raw + s * G_RAW, ta = tmem + G_A + n % G_A_BUFS * G_A_COLS + lanes;
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ld_shared_v4(src + ((j ^ (row & 7)) << 4));
        uint32_t r[2][32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t(&o)[32] = r[j >> 2];
          const int at = (j & 3) * 8;
          widen(v[j].x, o[at], o[at + 1]);
          widen(v[j].y, o[at + 2], o[at + 3]);
          widen(v[j].z, o[at + 4], o[at + 5]);
          widen(v[j].w, o[at + 6], o[at + 7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&rawempty[s]));
        const uint32_t before = n - G_A_BUFS;  // the step that had the buffer
        if (n >= G_A_BUFS && !warp_wait(smem_u32(&done[before % G_TOK_STAGES]), before / G_TOK_STAGES & 1u, c, W_EMPTY, 32, true)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st_32x32b_x32(ta, r[0]);
        tmem_st_32x32b_x32(ta + 32, r[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_light(mapa_shared(smem_u32(&full[n % G_TOK_STAGES]), 0u));
      }
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    int it = 0;
    for (int u = pair; u < units; u += pairs, ++it) {
      const Q8Unit w(p, u);
      const uint32_t b = it & 1;
      if (!warp_wait(smem_u32(&tfull[b]), static_cast<uint32_t>(it >> 1) & 1u, c, W_TFULL, b, true)) break;
      tc_fence_after();
      const int ch = w.ct * G_CH + static_cast<int>(cta) * G_ROWS + quarter * 32 + lane;
      const bool in = ch < p.a.N;
      const float ws = in ? load_global(p.a.w_scales + ch) : 0.0f;
      float bias = 0.0f;
      if (in && p.a.bias != nullptr) {
        const uint16_t h = load_global(static_cast<const uint16_t*>(p.a.bias) + ch);
        bias = DT == 1 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
      }
      const int t0 = w.tt * p.n;
      for (int c0 = 0; c0 < p.n && t0 + c0 < p.a.M; c0 += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem + b * G_TOK + c0 + (static_cast<uint32_t>(quarter * 32) << 16), r);
        const int left = min(16, p.a.M - t0 - c0);
        if (p.parts != nullptr) {
          float* dst = p.parts + (static_cast<size_t>(w.split) * p.a.M + t0 + c0) * p.a.N + ch;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (in && j < left) dst[static_cast<size_t>(j) * p.a.N] = __uint_as_float(r[j]);
        } else {
          const float xs = (lane & 15) < left ? load_global(p.a.x_scales + t0 + c0 + (lane & 15)) : 0.0f;
          uint16_t* dst = static_cast<uint16_t*>(p.a.out) + static_cast<size_t>(t0 + c0) * p.a.N + ch;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float v = __uint_as_float(r[j]) * __shfl_sync(0xFFFFFFFFu, xs, j) * ws + bias;
            if (in && j < left) dst[static_cast<size_t>(j) * p.a.N] = static_cast<uint16_t>(pack2<DT>(v, 0.0f));
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
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

// Adds the parts of K, four channels a thread.
template <int DT>
__global__ void __launch_bounds__(256) q8_parts_kernel(const __grid_constant__ Q8Args a, const float* parts, int splits) {
  after_previous();
  const size_t n4 = static_cast<size_t>(a.M) * a.N / 4, i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4* src = reinterpret_cast<const float4*>(parts) + i;
  float4 s = __ldcg(src);
  for (int k = 1; k < splits; ++k) {
    const float4 o = __ldcg(src + k * n4);
    s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
  }
  const int row = static_cast<int>(4 * i / a.N), ch = static_cast<int>(4 * i - static_cast<size_t>(row) * a.N);
  const float xs = load_global(a.x_scales + row);
  const float4 ws = load_global(reinterpret_cast<const float4*>(a.w_scales + ch));
  float b[4] = {};
  if (a.bias != nullptr) {
    const uint2 h = load_global(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.bias) + ch));
    const uint16_t e[4] = {static_cast<uint16_t>(h.x), static_cast<uint16_t>(h.x >> 16), static_cast<uint16_t>(h.y), static_cast<uint16_t>(h.y >> 16)};
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = DT == 1 ? __uint_as_float(static_cast<uint32_t>(e[j]) << 16) : __half2float(__ushort_as_half(e[j]));
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + 4 * i) =
      make_uint2(pack2<DT>(s.x * xs * ws.x + b[0], s.y * xs * ws.y + b[1]), pack2<DT>(s.z * xs * ws.z + b[2], s.w * xs * ws.w + b[3]));
}

constexpr int G_MOST_SPLITS = 16, G_MOST_UNITS = 4 * G_PAIRS;  // parts of K; units where K is cut

// Tokens of a tile and parts of K: those of the least estimated time, in cycles.  A step
// of n tokens takes 4 n cycles of products, and at least as long as the weights' bytes
// need; a unit begins and ends with about 1500 cycles that nothing covers, and the
// parts are written and read again at some 5 KB a cycle.
struct Q8Plan {
  int n, tok_tiles, ch_tiles, steps, splits;
  size_t x_bytes, part_bytes;
};

Q8Plan q8_plan(int M, int N, int K) {
  Q8Plan best{};
  best.ch_tiles = ceil_div(N, G_CH);
  best.steps = ceil_div(K, G_K);
  double least = 0.0;
  const int fewest = ceil_div(M, G_TOK);
  for (int most = G_TOK; most > 0; most -= 16) {
    const int tt = ceil_div(M, most), n = ceil_div(ceil_div(M, tt), 16) * 16;
    if (tt > fewest + fewest / 2 + 1) break;
    const double step = std::max(4.0 * n, 600.0);
    for (int splits = 1; splits <= G_MOST_SPLITS && splits <= best.steps; ++splits) {
      const long long units = static_cast<long long>(tt) * best.ch_tiles * splits;
      if (splits > 1 && units > G_MOST_UNITS) break;
      const double waves = static_cast<double>((units + G_PAIRS - 1) / G_PAIRS);
      double time = waves * (ceil_div(best.steps, splits) * step + 1500.0);
      if (splits > 1) time += 3000.0 + 8.0 * splits * M * N / 5000.0;
      if (least == 0.0 || time < least) {
        least = time;
        best.n = n;
        best.tok_tiles = tt;
        best.splits = splits;
      }
    }
  }
  // whole tiles: what lies past the last token is read, and never stored
  best.x_bytes = round_up(static_cast<size_t>(best.n) * best.tok_tiles * K * 2, WS_ALIGN);
  best.part_bytes = best.splits > 1 ? sizeof(float) * best.splits * M * N : 0;
  return best;
}

template <int DT>
flux_status_t launch(const Q8GemmParams& p, const DeviceInfo& dev, cudaStream_t s) {
  constexpr auto kernel = q8_gemm_kernel<DT>;
  static OncePerDevice once;
  cudaError_t e = once(dev.device, [] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM); });
  if (e != cudaSuccess) return cuda_fail(e);
  const long long units = static_cast<long long>(p.ch_tiles) * p.tok_tiles * p.splits;
  const unsigned grid = static_cast<unsigned>(2 * std::min<long long>(std::min(dev.sm_count / 2, G_PAIRS), units));
  e = launch_after(kernel, grid, G_THREADS, G_SMEM, 2, s, p);
  if (e == cudaSuccess && p.parts != nullptr) {
    const size_t n4 = static_cast<size_t>(p.a.M) * p.a.N / 4;
    e = launch_after(q8_parts_kernel<DT>, static_cast<unsigned>((n4 + 255) / 256), 256, 0, 1, s, p.a, p.parts, p.splits);
  }
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

}  // namespace

size_t q8_gemm_bytes(int M, int N, int K) {
  const Q8Plan p = q8_plan(M, N, K);
  return p.x_bytes + p.part_bytes;
}

// Enough for every call of up to M rows: up to 15 rows of padding a tile, and the parts
// of as many units as are cut at most.
size_t q8_gemm_most_bytes(int M, int N, int K) {
  const int fewest = ceil_div(M, G_TOK);
  const size_t rows = static_cast<size_t>(M) + 16 * (static_cast<size_t>(fewest) + fewest / 2 + 1);
  const size_t parts = std::min(sizeof(float) * G_MOST_SPLITS * M * N, sizeof(float) * G_MOST_UNITS * G_CH * G_TOK);
  return round_up(rows * K * 2, WS_ALIGN) + parts;
}

flux_status_t q8_gemm_launch(const Q8Args& a, flux_dtype_t dtype, void* workspace, const DeviceInfo& dev, cudaStream_t s) {
  const Q8Plan plan = q8_plan(a.M, a.N, a.K);
  if (static_cast<long long>(plan.ch_tiles) * plan.tok_tiles * plan.splits > INT_MAX) return FLUX_ERR_UNSUPPORTED;
  char* at = static_cast<char*>(workspace) + WS_HEADER;
  const size_t nx = static_cast<size_t>(a.M) * a.K / 16;
  const unsigned blocks = static_cast<unsigned>(std::min<size_t>((nx + 255) / 256, static_cast<size_t>(dev.sm_count) * 8));
  const cudaError_t e = launch_after(q8_widen_kernel, blocks, 256, 0, 1, s, reinterpret_cast<const uint4*>(a.x), reinterpret_cast<uint4*>(at), nx);
  if (e != cudaSuccess) return cuda_fail(e);
  Q8GemmParams p{};
  flux_status_t st = encode_2d(&p.x, FLUX_F16, at, a.K, static_cast<uint64_t>(plan.n) * plan.tok_tiles, a.K * 2ull, 64, plan.n / 2);
  if (st == FLUX_OK) st = encode_2d_u8(&p.w, a.w, a.K, a.N, a.K, G_K, G_ROWS);
  if (st != FLUX_OK) return st;
  p.a = a;
  p.parts = plan.splits > 1 ? reinterpret_cast<float*>(at + plan.x_bytes) : nullptr;
  p.hdr = static_cast<uint32_t*>(workspace);
  p.seq = next_seq();
  p.timeout_ns = DEFAULT_TIMEOUT_NS;
  p.n = plan.n;
  p.ch_tiles = plan.ch_tiles;
  p.tok_tiles = plan.tok_tiles;
  p.steps = plan.steps;
  p.splits = plan.splits;
  return dtype == FLUX_BF16 ? launch<1>(p, dev, s) : launch<0>(p, dev, s);
}

}  // namespace flux
