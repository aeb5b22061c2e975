// Products of few rows with 4-bit weights: out = x . W, W[k, n] = scale[k / group, n] (code[n, k] - 8).
//
// With a handful of rows such a product does 2 M operations per half byte of
// weights, so it is bound by reading the weights once.  They are stored
// column by column, 128 inputs (64 bytes) at a time, in the order in which
// the lanes of a warp use them: in each run of 128 inputs, 16 bytes for every
// c of 0..3, in them one 32-bit word for every j of 0..3, whose nibbles i and
// i + 4 hold the inputs 32 j + 8 c + 2 i and 32 j + 8 c + 2 i + 1.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "flux_host.h"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int W4_RUN = 128;  // inputs per run of 64 bytes

enum W4Mode { W4_DENSE = 0, W4_LAYER0 = 1, W4_LAYER1 = 2 };

constexpr int W4_WARPS = 8, W4_THREADS = W4_WARPS * 32;
constexpr int W4_COLS = W4_WARPS * 16;      // columns of a tile: 16 for each warp
constexpr int W4_MAX_CTAS = 3 * 160;        // at most three CTAs per SM
constexpr int W4_RUN_BYTES = W4_RUN / 2;

struct W4Args {
  const uint16_t* x;
  const uint8_t* q;
  const uint16_t* scales;
  const int32_t* ids;
  const float* weights;
  uint16_t* out;
  uint32_t* hdr;
  uint32_t* cut;        // [grid] arrivals at the tile that CTA i is the first of several to work on
  uint32_t* done;       // [column tiles] layer1: finished row tiles
  float* parts;         // [2 grid] partial tiles: of each CTA's first and last
  float* rows_f32;      // layer1: [slots x N]
  int slots;            // rows of x . W: M, or T topk
  int T, N, K, runs, group, groups, E, topk, mode;
};

// Rows of one expert that one tile multiplies.
struct W4RowTile {
  uint16_t expert, first, rows;  // `rows` entries of the slot order from `first`
};

// 16 x 8 += 16 x 16 . 16 x 8; A four and B two registers of two 16-bit values.
template <int DT>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  if constexpr (DT == 1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// (v & mask) | bits
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}

// The eight codes of a word less 8 as pairs of 16-bit values: nibbles i and
// i + 4 in pair i.  A code in the low bits of a power of two's significand is
// that power plus the code; the difference is exact.
template <int DT>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&p)[4]) {
  if constexpr (DT == 1) {
    const __nv_bfloat162 bias = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u);  // 128 + code
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), bias);
      p[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
  } else {
    const __half2 bias = __floats2half2_rn(1032.0f, 1032.0f), sixteenth = __floats2half2_rn(0.0625f, 0.0625f),
                  bias16 = __floats2half2_rn(-72.0f, -72.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w >> (8 * i);
      const uint32_t lo = and_or(v, 0x000F000Fu, 0x64006400u);  // 1024 + code
      const uint32_t hi = and_or(v, 0x00F000F0u, 0x64006400u);  // 1024 + 16 code
      const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
      const __half2 b = __hfma2(*reinterpret_cast<const __half2*>(&hi), sixteenth, bias16);
      p[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
      p[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
}

// 16 bytes to shared memory, or zeros where `take` is false.
__device__ __forceinline__ void copy16_or_zero(void* smem, const void* gmem, bool take) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(gmem), "r"(take ? 16 : 0) : "memory");
}

// MT tiles of 8 rows; SR scales per run and column (a group of 128 or a multiple: 1, of 64: 2, else 4).
template <int MT, int SR>
struct W4Shape {
  static constexpr int CHUNK = MT == 1 ? 24 : MT == 2 ? 16 : 8;  // runs whose rows of x and scales are in shared memory
  static constexpr int XRUN = MT * 8 * W4_RUN * 2;
  static constexpr int SRUN = SR * W4_COLS * 2;
  static constexpr int SMEM = CHUNK * (XRUN + SRUN);
  static constexpr int AHEAD = 4;                // runs of codes that a thread has on the way
  static constexpr int CTAS = 2;                 // per SM
  static constexpr int PART = W4_COLS * MT * 8;  // floats of a partial tile
};

// out = x . W for few rows.  The work is units of one tile of 128 columns, up
// to 8 MT rows of one expert, and one run of 128 inputs; unit ids count the
// runs of a tile, then the column tiles, then the row tiles, and every CTA
// takes an equal stretch of them, so a tile may be cut between CTAs.
//
// A warp multiplies 16 columns: the codes are the A operand of 16 x 8 x 16
// tensor instructions, the rows of x the B operand (a matrix-vector product
// leaves 7 of its 8 columns idle, which costs nothing: the kernel is bound by
// the bytes of the codes and by the instructions that unpack them).  Every
// thread copies the words that it will unpack itself; rows of x and scales are
// shared by the CTA, in a ring of STAGES runs with one barrier per run.
//
// The sums of a group are exact products in fp32, then scaled into the tile's
// sums.  The CTAs that share a tile leave their sums in the workspace, and the
// last to arrive adds them in CTA order: repeat calls give the same bits.
template <int DT, int MT, int SR>
__global__ void __launch_bounds__(W4_THREADS, (W4Shape<MT, SR>::CTAS)) w4_kernel(const __grid_constant__ W4Args a) {
  using S = W4Shape<MT, SR>;
  extern __shared__ uint4 ring4[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(ring4);
  __shared__ uint16_t order[FLUX_W4_MAX_ROWS];       // slots by expert
  __shared__ W4RowTile tiles[FLUX_W4_MAX_ROWS];
  int* hist = reinterpret_cast<int*>(ring);  // before the ring is used
  __shared__ int scan[2][W4_WARPS];
  __shared__ int last_here;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int col_tiles = (a.N + W4_COLS - 1) / W4_COLS;
  int row_tiles;
  if (a.mode == W4_DENSE) {
    row_tiles = (a.slots + MT * 8 - 1) / (MT * 8);
    for (int i = tid; i < row_tiles; i += W4_THREADS)
      tiles[i] = W4RowTile{0, static_cast<uint16_t>(i * MT * 8), static_cast<uint16_t>(min(MT * 8, a.slots - i * MT * 8))};
    for (int i = tid; i < a.slots; i += W4_THREADS) order[i] = static_cast<uint16_t>(i);
    __syncthreads();
  } else {
    // stable counting sort of the slots by expert: CTAs that share a tile have to
    // agree on the order of its rows
    for (int e = tid; e < a.E; e += W4_THREADS) hist[e] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < a.slots; i += W4_THREADS) {
      const int e = a.ids[i];
      if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
      else bad = true;
    }
    if (bad) atomicCAS(a.hdr, 0u, static_cast<uint32_t>(FLUX_ERR_INVALID_ARG));
    __syncthreads();
    // exclusive sums of slots and row tiles; thread i has the experts 4 i .. 4 i + 3
    int n[4], slots = 0, rt = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = tid * 4 + k;
      n[k] = e < a.E ? hist[e] : 0;
      slots += n[k];
      rt += (n[k] + MT * 8 - 1) / (MT * 8);
    }
    int s0 = slots, r0 = rt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int s1 = __shfl_up_sync(0xFFFFFFFFu, s0, o), r1 = __shfl_up_sync(0xFFFFFFFFu, r0, o);
      if (lane >= o) {
        s0 += s1;
        r0 += r1;
      }
    }
    if (lane == 31) {
      scan[0][warp] = s0;
      scan[1][warp] = r0;
    }
    __syncthreads();
    s0 -= slots;
    r0 -= rt;
    row_tiles = 0;
#pragma unroll
    for (int w = 0; w < W4_WARPS; ++w) {
      if (w < warp) {
        s0 += scan[0][w];
        r0 += scan[1][w];
      }
      row_tiles += scan[1][w];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = tid * 4 + k;
      if (e < a.E) hist[e] = s0;
      for (int m = 0; m < n[k]; m += MT * 8)
        tiles[r0++] = W4RowTile{static_cast<uint16_t>(e), static_cast<uint16_t>(s0 + m),
                                static_cast<uint16_t>(min(MT * 8, n[k] - m))};
      s0 += n[k];
    }
    __syncthreads();
    if (warp == 0) {
      for (int i0 = 0; i0 < a.slots; i0 += 32) {
        const int i = i0 + lane, e = i < a.slots ? a.ids[i] : -1;
        const bool in = e >= 0 && e < a.E;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, in ? e : -1 - lane);
        const int at = in ? hist[e] : 0;
        __syncwarp();
        if (in) {
          order[at + __popc(same & ((1u << lane) - 1u))] = static_cast<uint16_t>(i);
          if (lane == __ffs(same) - 1) hist[e] = at + __popc(same);
        }
        __syncwarp();
      }
    }
    __syncthreads();
    if (a.mode == W4_LAYER0) {  // slots of no expert
      for (int i = blockIdx.x; i < a.slots; i += gridDim.x) {
        const int e = a.ids[i];
        if (e < 0 || e >= a.E)
          for (int k = tid * 8; k < a.N; k += W4_THREADS * 8)
            *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(i) * a.N + k) = make_uint4(0, 0, 0, 0);
      }
    } else if (row_tiles == 0) {
      for (size_t k = (static_cast<size_t>(blockIdx.x) * W4_THREADS + tid) * 8; k < static_cast<size_t>(a.T) * a.N;
           k += static_cast<size_t>(gridDim.x) * W4_THREADS * 8)
        *reinterpret_cast<uint4*>(a.out + k) = make_uint4(0, 0, 0, 0);
    }
  }

  const int units = row_tiles * col_tiles * a.runs;
  // every CTA that works has a unit: the arrivals at a cut tile are counted by CTA
  const int ctas = min(static_cast<int>(gridDim.x), units), me = blockIdx.x;
  if (me >= ctas) return;
  const int each = units / ctas, more = units - each * ctas;  // the first `more` CTAs have one unit more
  auto first_unit = [&](int cta) { return cta * each + min(cta, more); };
  auto cta_of = [&](int unit) {
    const int big = more * (each + 1);
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  };
  const int u0 = first_unit(me), n_units = first_unit(me + 1) - u0;
  int tile = u0 / a.runs, run = u0 - tile * a.runs;

  const int x_from0 = g * 256 + c * 16 + ((g & 1) << 6), x_from1 = x_from0 ^ 64;
  constexpr int P = S::AHEAD;
  constexpr int XROWS = MT == 1 ? 8 : 16, XRUNS = 16 / XROWS;  // rows and runs of x that the CTA copies at a time
  int todo = n_units;
#pragma unroll 1
  for (bool first_tile = true; todo > 0; ++tile, run = 0, first_tile = false) {
    const int n_runs = min(a.runs - run, todo);
    const bool whole = n_runs == a.runs;
    todo -= n_runs;
    const int rt_i = tile / col_tiles, ct = tile - rt_i * col_tiles, col0 = ct * W4_COLS;
    const W4RowTile rt = tiles[rt_i];
    // this thread's words of the columns g and g + 8 of the warp's 16
    const int my_col = col0 + warp * 16 + g;
    const uint4* qa = reinterpret_cast<const uint4*>(
        a.q + ((static_cast<size_t>(rt.expert) * a.N + min(my_col, a.N - 1)) * a.runs + run) * W4_RUN_BYTES + c * 16);
    const uint4* qb = reinterpret_cast<const uint4*>(
        a.q + ((static_cast<size_t>(rt.expert) * a.N + min(my_col + 8, a.N - 1)) * a.runs + run) * W4_RUN_BYTES + c * 16);
    uint4 wa[P], wb[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i < n_runs) {
        wa[i] = __ldcs(qa + i * 4);
        wb[i] = __ldcs(qb + i * 4);
      }
    }
    float acc[MT][4] = {};
#pragma unroll 1
    for (int r0 = 0; r0 < n_runs; r0 += S::CHUNK) {
      const int n = min(S::CHUNK, n_runs - r0);
      __syncthreads();  // the last chunk has been read
      // rows of x in 16-byte chunks (8 inputs): chunk 4 j + c of a row lies at
      // 4 (j ^ (row & 1)) + c, so that two rows' reads meet different banks
      {
        const int k = tid & 15, k0 = (run + r0) * W4_RUN + k * 8;
#pragma unroll
        for (int p = 0; p < (MT * 8 + 15) / 16; ++p) {
          const int m = p * 16 + (tid >> 4) % XROWS;
          if (m < rt.rows) {
            const int slot = order[rt.first + m];
            const uint16_t* row = a.x + static_cast<size_t>(a.mode == W4_LAYER0 ? slot / a.topk : slot) * a.K;
            uint8_t* to = ring + m * 256 + ((k ^ ((m & 1) << 2)) << 4);
#pragma unroll 4
            for (int r = (tid >> 4) / XROWS; r < n; r += XRUNS) {
              const int at = k0 + r * W4_RUN;
              copy16_or_zero(to + r * S::XRUN, row + (at < a.K ? at : 0), at < a.K);
            }
          }
        }
        constexpr int AT_ONCE = W4_THREADS / (SR * W4_COLS / 8);
        const int sr = tid / (W4_COLS / 8) % SR, col = tid % (W4_COLS / 8) * 8;
        for (int r = tid / (SR * W4_COLS / 8); r < n; r += AT_ONCE) {
          const int at = (run + r0 + r) * W4_RUN + sr * (W4_RUN / SR);
          const bool in = at < a.K && col0 + col < a.N;
          const size_t from = (static_cast<size_t>(rt.expert) * a.groups + (in ? at / a.group : 0)) * a.N + (in ? col0 + col : 0);
          copy16_or_zero(ring + S::CHUNK * S::XRUN + r * S::SRUN + (sr * W4_COLS + col) * 2, a.scales + from, in);
        }
        copy_commit();
        copy_wait<0>();
      }
      __syncthreads();
      const uint8_t* xs = ring;
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(ring + S::CHUNK * S::XRUN) + warp * 16 + g;
#pragma unroll 1
      for (int r = 0; r < n; r += P, xs += P * S::XRUN, sc += P * S::SRUN / 2, qa += P * 4, qb += P * 4) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (r + i >= n) break;
          const uint32_t va[4] = {wa[i].x, wa[i].y, wa[i].z, wa[i].w}, vb[4] = {wb[i].x, wb[i].y, wb[i].z, wb[i].w};
          if (r0 + r + i + P < n_runs) {
            wa[i] = __ldcs(qa + (i + P) * 4);
            wb[i] = __ldcs(qb + (i + P) * 4);
          }
          float part[MT][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t pa[4], pb[4];
            codes8<DT>(va[j], pa);
            codes8<DT>(vb[j], pb);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if (m == 0 || rt.rows > m * 8) {
                const uint4 xv = *reinterpret_cast<const uint4*>(xs + i * S::XRUN + (j & 1 ? x_from1 : x_from0) + (j >> 1) * 128 + m * 2048);
                if (j % (4 / SR) == 0) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) part[m][k] = 0.0f;
                }
                mma_16x8x16<DT>(part[m], pa[0], pb[0], pa[1], pb[1], xv.x, xv.y);
                mma_16x8x16<DT>(part[m], pa[2], pb[2], pa[3], pb[3], xv.z, xv.w);
              }
            }
            if ((j + 1) % (4 / SR) == 0) {
              const uint16_t* s = sc + i * (S::SRUN / 2) + j / (4 / SR) * W4_COLS;
              const float s0 = unpack2<DT>(s[0]).x, s1 = unpack2<DT>(s[8]).x;
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                if (m == 0 || rt.rows > m * 8) {
                  acc[m][0] += s0 * part[m][0];
                  acc[m][1] += s0 * part[m][1];
                  acc[m][2] += s1 * part[m][2];
                  acc[m][3] += s1 * part[m][3];
                }
              }
            }
          }
        }
      }
    }

    if (!whole) {
      // leave the sums; the last CTA of the tile adds everybody's
      const int place = 2 * me + (first_tile ? 0 : 1);
      float4* mine = reinterpret_cast<float4*>(a.parts + static_cast<size_t>(place) * S::PART);
#pragma unroll
      for (int m = 0; m < MT; ++m) mine[m * W4_THREADS + tid] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
      __threadfence();
      __syncthreads();
      const int tu0 = tile * a.runs, c0 = cta_of(tu0), c1 = cta_of(tu0 + a.runs - 1);
      if (tid == 0) {
        const uint32_t seen = atomicAdd(a.cut + c0, 1u);
        last_here = seen == static_cast<uint32_t>(c1 - c0);
        if (last_here) a.cut[c0] = 0u;
      }
      __syncthreads();
      if (!last_here) continue;
      __threadfence();
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
      constexpr int BATCH = MT == 1 ? 4 : 2;  // CTAs whose loads are in flight together
      for (int k0 = c0; k0 <= c1; k0 += BATCH) {
        float4 v[BATCH][MT];
        float4* p[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int k = k0 + b;
          if (k > c1) break;
          // the tile is the first of CTA k unless it begins inside its stretch
          p[b] = reinterpret_cast<float4*>(a.parts + static_cast<size_t>(2 * k + (first_unit(k) >= tu0 ? 0 : 1)) * S::PART);
#pragma unroll
          for (int m = 0; m < MT; ++m) v[b][m] = __ldcg(p[b] + m * W4_THREADS + tid);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          if (k0 + b > c1) break;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            p[b][m * W4_THREADS + tid] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            acc[m][0] += v[b][m].x;
            acc[m][1] += v[b][m].y;
            acc[m][2] += v[b][m].z;
            acc[m][3] += v[b][m].w;
          }
        }
      }
    }
    // columns g and g + 8 of the warp's 16, rows 2 c and 2 c + 1 of every eight
    const int col = ct * W4_COLS + warp * 16 + g;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = m * 8 + 2 * c + (i & 1), n = col + (i >> 1) * 8;
        if (r < rt.rows && n < a.N) {
          const size_t at = static_cast<size_t>(order[rt.first + r]) * a.N + n;
          if (a.mode == W4_LAYER1) a.rows_f32[at] = acc[m][i];
          else a.out[at] = static_cast<uint16_t>(pack2<DT>(acc[m][i], 0.0f));
        }
      }
    }
    if (a.mode != W4_LAYER1) continue;
    // the last row tile of these columns adds the slots of every token
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      last_here = atomicAdd(a.done + ct, 1u) == static_cast<uint32_t>(row_tiles - 1);
      if (last_here) a.done[ct] = 0u;
    }
    __syncthreads();
    if (!last_here) continue;
    __threadfence();
    const int cols = min(W4_COLS, a.N - ct * W4_COLS);
    for (int i = tid; i < a.T * (W4_COLS / 4); i += W4_THREADS) {
      const int t = i / (W4_COLS / 4), n = i % (W4_COLS / 4) * 4;
      if (n >= cols) continue;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k0 = 0; k0 < a.topk; k0 += 8) {
        float4 v[8];
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int slot = t * a.topk + k0 + k;
          const int e = k0 + k < a.topk ? a.ids[slot] : -1;
          const bool in = e >= 0 && e < a.E;
          w[k] = in ? a.weights[slot] : 0.0f;
          v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (in) v[k] = __ldcg(reinterpret_cast<const float4*>(a.rows_f32 + static_cast<size_t>(slot) * a.N + ct * W4_COLS + n));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k0 + k < a.topk)
            *reinterpret_cast<float4*>(a.rows_f32 + static_cast<size_t>(t * a.topk + k0 + k) * a.N + ct * W4_COLS + n) =
                make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          s.x += w[k] * v[k].x;
          s.y += w[k] * v[k].y;
          s.z += w[k] * v[k].z;
          s.w += w[k] * v[k].w;
        }
      }
      *reinterpret_cast<uint2*>(a.out + static_cast<size_t>(t) * a.N + ct * W4_COLS + n) =
          make_uint2(pack2<DT>(s.x, s.y), pack2<DT>(s.z, s.w));
    }
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

// Workspace: header, arrivals, finished row tiles, partial tiles, fp32 rows.
struct W4Ws {
  size_t cut, done, parts, rows, total;
};

int w4_row_tiles_of_8(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

W4Ws w4_ws(int slots, int N) {
  W4Ws w{};
  size_t at = WS_HEADER;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, WS_ALIGN);
    return here;
  };
  w.cut = take(sizeof(uint32_t) * W4_MAX_CTAS);
  w.done = take(sizeof(uint32_t) * ((N + W4_COLS - 1) / W4_COLS));
  w.parts = take(sizeof(float) * 2 * W4_MAX_CTAS * W4_COLS * 8 * w4_row_tiles_of_8(slots));
  w.rows = take(sizeof(float) * slots * static_cast<size_t>(N));
  w.total = at;
  return w;
}

template <int DT, int MT, int SR>
flux_status_t w4_launch(const W4Args& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int smem = W4Shape<MT, SR>::SMEM;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(w4_kernel<DT, MT, SR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr != cudaSuccess) return cuda_fail(attr);
  // no more CTAs than units (of as many row tiles as the slots can make)
  const long long col_tiles = (a.N + W4_COLS - 1) / W4_COLS;
  const long long row_tiles = a.mode == W4_DENSE ? (a.slots + MT * 8 - 1) / (MT * 8) : a.slots;
  const long long units = row_tiles * col_tiles * a.runs;
  if (units > INT_MAX) return FLUX_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(std::min<long long>(units, std::min(W4Shape<MT, SR>::CTAS * dev.sm_count, W4_MAX_CTAS)));
  w4_kernel<DT, MT, SR><<<grid, W4_THREADS, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
}

template <int DT, int MT>
flux_status_t w4_launch_groups(const W4Args& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.group % W4_RUN == 0) return w4_launch<DT, MT, 1>(a, dev, s);
  if (a.group == W4_RUN / 2) return w4_launch<DT, MT, 2>(a, dev, s);
  return w4_launch<DT, MT, 4>(a, dev, s);
}

template <int DT>
flux_status_t w4_launch_rows(const W4Args& a, const DeviceInfo& dev, cudaStream_t s) {
  // the most rows one expert can have
  const int mt = w4_row_tiles_of_8(a.mode == W4_DENSE ? a.slots : a.T);
  if (mt == 1) return w4_launch_groups<DT, 1>(a, dev, s);
  if (mt == 2) return w4_launch_groups<DT, 2>(a, dev, s);
  return w4_launch_groups<DT, 4>(a, dev, s);
}

bool w4_common_ok(int N, int K, int group, int E, flux_dtype_t dtype) {
  return N >= 0 && K >= 0 && group >= 1 && E >= 1 && E <= FLUX_MAX_EXPERTS && (dtype == FLUX_F16 || dtype == FLUX_BF16);
}

flux_status_t w4_run(W4Mode mode, int rows, int slots, int T, int N, int K, int E, int topk, int group,
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
  flux_status_t st = check_workspace(workspace, workspace_bytes, flux_w4_workspace_size(slots, N, K, E));
  if (st != FLUX_OK) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FLUX_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    const cudaError_t e = cudaMemsetAsync(out, 0, sizeof(uint16_t) * rows * static_cast<size_t>(N), s);
    return e == cudaSuccess ? FLUX_OK : cuda_fail(e);
  }
  const W4Ws w = w4_ws(slots, N);
  char* ws = static_cast<char*>(workspace);
  W4Args a{};
  a.x = static_cast<const uint16_t*>(x);
  a.q = static_cast<const uint8_t*>(q);
  a.scales = static_cast<const uint16_t*>(scales);
  a.ids = ids;
  a.weights = weights;
  a.out = static_cast<uint16_t*>(out);
  a.hdr = static_cast<uint32_t*>(workspace);
  a.cut = reinterpret_cast<uint32_t*>(ws + w.cut);
  a.done = reinterpret_cast<uint32_t*>(ws + w.done);
  a.parts = reinterpret_cast<float*>(ws + w.parts);
  a.rows_f32 = reinterpret_cast<float*>(ws + w.rows);
  a.slots = slots;
  a.T = T;
  a.N = N;
  a.K = K;
  a.runs = (K + W4_RUN - 1) / W4_RUN;
  a.group = group;
  a.groups = (K + group - 1) / group;
  a.E = E;
  a.topk = topk;
  a.mode = mode;
  return dtype == FLUX_BF16 ? w4_launch_rows<1>(a, dev, s) : w4_launch_rows<0>(a, dev, s);
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
  return w4_ws(rows, N).total;
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
