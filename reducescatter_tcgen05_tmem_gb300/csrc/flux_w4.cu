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
#include <type_traits>

#include "flux_host.h"
#include "flux_ptx.cuh"
#include "flux_rows.cuh"

namespace flux {

namespace {

constexpr int W4_RUN = 128;  // inputs per run of 64 bytes

enum W4Mode { W4_DENSE = 0, W4_LAYER0 = 1, W4_LAYER1 = 2 };

constexpr int W4_WARPS = 4, W4_THREADS = W4_WARPS * 32;  // of a team
constexpr int W4_CA = 2;                         // A operands (16 columns each) of a warp
constexpr int W4_COLS = W4_WARPS * 16 * W4_CA;   // columns of a tile
constexpr int W4_MIN_UNITS = 4;
constexpr int W4_MAX_TEAMS = 4 * 160;            // at most four per SM
constexpr int W4_RUN_BYTES = W4_RUN / 2;
constexpr int W4_MAX_SIZE = INT_MAX - 1023;      // of N and K: rounded up to tiles, runs and blocks they still are ints
constexpr int W4_NONE = 0xFFFF;                  // row tile of a slot whose expert id is out of range

// Equal stretches of units: team i has the units [first(i), first(i + 1)).
struct W4Split {
  int each, more;  // the first `more` teams have one unit more
  __device__ __forceinline__ int first(int team) const { return team * each + min(team, more); }
  __device__ __forceinline__ int team_of(int unit) const {
    const int big = more * (each + 1);
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  }
};

// Where a slot's sums are: its row tile (W4_NONE: nowhere) and its row in it.
struct W4Slot {
  uint16_t tile, row;
};

struct W4Args {
  const uint16_t* x;
  const uint8_t* q;
  const uint16_t* scales;
  const int32_t* ids;
  const float* weights;
  uint16_t* out;
  uint32_t* hdr;
  // how the products' kernel cut its units, for the one that joins them: known to
  // the host (dense) or left in the workspace
  W4Split dense_split;
  W4Split* split;
  W4Slot* where;        // [slots]
  uint32_t* joined;     // blocks of the joining kernel that are done with those
  float* parts;         // [2 teams] sums of cut tiles: of each team's first and last
  float* rows_f32;      // layer1: [slots x N]
  int slots;            // rows of x . W: M, or T topk
  int T, N, K, runs, group, groups, E, topk, mode, teams;
};

// Rows of one expert that one tile multiplies.
struct W4RowTile {
  uint16_t expert, first, rows;  // `rows` entries of the slot order from `first`
};

// d (+)= 16 x 16 . 16 x 8; A four and B two registers of two 16-bit values.
template <int DT, bool FROM_ZERO>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  const float c0 = FROM_ZERO ? 0.0f : d[0], c1 = FROM_ZERO ? 0.0f : d[1], c2 = FROM_ZERO ? 0.0f : d[2],
              c3 = FROM_ZERO ? 0.0f : d[3];
  if constexpr (DT == 1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
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
// that power plus the code; the difference is exact (the method is published, in
// Kim et al., "Who Says Elephants Can't Run", 2022).
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

__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
// Codes are read once, 64 bytes of a column at a time; the hint has L2 fetch the
// next runs of the column with them.
__device__ __forceinline__ uint4 load_codes(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Scales of four columns, each twice for the two rows it multiplies.
template <int DT>
__device__ __forceinline__ void shared_scales(uint32_t at, f32x2 (&s)[4]) {
  uint32_t lo, hi;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(at));
  const float2 a = unpack2<DT>(lo), b = unpack2<DT>(hi);
  s[0] = both(a.x), s[1] = both(a.y), s[2] = both(b.x), s[3] = both(b.y);
}

// 16 bytes to shared memory, or zeros where `take` is false.
__device__ __forceinline__ void copy16_or_zero(void* smem, const void* gmem, bool take) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(gmem), "r"(take ? 16 : 0) : "memory");
}

// MT tiles of 8 rows; SR scales per run and column (a group of 128 or a multiple: 1, of 64: 2, else 4).
template <int MT, int SR>
struct W4Shape {
  // Warps of a scheduler come forward by age: of an SM's four CTAs of one team the
  // first is done with its stretch after 25 us and the last after 36.  In a CTA of
  // four teams whose four warps have four different ages all end within 3 us (layer1
  // of 24 tokens, 6 of 64 experts, 1792 x 4096: 69 -> 66 us; one row of 4096 x 4096
  // 8.9 -> 8.3).  Three teams that way are slower than three CTAs (13 rows of
  // 28672 x 8192: 39.0 us, 37.4).
  static constexpr int TEAMS = MT == 1 ? 4 : 1;                  // of a CTA
  static constexpr int CTAS = MT == 4 ? 2 : MT == 2 ? 3 : 1;     // per SM
  static constexpr int THREADS = TEAMS * W4_THREADS;
  static constexpr int AHEAD = 2;                               // runs of codes that a thread has on the way
  static constexpr int CHUNK = MT == 1 ? 6 : MT == 2 ? 4 : 2;   // runs whose rows of x and scales make one buffer
  static_assert(CHUNK % AHEAD == 0, "the words on the way keep their places from one buffer to the next");
  static constexpr int XRUN = MT * 8 * W4_RUN * 2;
  static constexpr int SRUN = SR * W4_COLS * 2;
  static constexpr int BUFFER = CHUNK * (XRUN + SRUN);
  static constexpr int SMEM = 2 * BUFFER;
  static constexpr int PART = W4_COLS * MT * 8;  // floats of a cut tile's sums
};

// out = x . W for few rows.  The work is units of one tile of 128 columns, up
// to 8 MT rows of one expert, and one run of 128 inputs; unit ids count the
// runs of a tile, then the column tiles, then the row tiles, and every team of
// four warps takes an equal stretch of them, so a tile may be cut between teams.
//
// A warp multiplies 32 columns: the codes are two A operands of 16 x 8 x 16
// tensor instructions, the rows of x the B operand (a matrix-vector product
// leaves 7 of its 8 columns idle, which costs nothing: the kernel is bound by
// the bytes of the codes and by the instructions that unpack them).  Every
// thread loads the words that it will unpack itself, AHEAD runs ahead; rows of
// x and scales are shared by the team, in two buffers of CHUNK runs, one filled
// while the other is used.
//
// The sums of a group are exact products in fp32, then scaled into the tile's
// sums.  Teams that share a tile leave their sums in the workspace, where
// w4_join_kernel adds them in team order: repeat calls give the same bits.
//
// With the joining kernel, a call in a row of calls: 1 row of 4096 x 4096 8.3 us
// (latency); 5 experts of 4096 x 14336 for 4 tokens 38 us, 4.0 TB/s over the call
// and 4.5 while it streams (issue slots 55 %, tensor pipe 22 %); 13 rows of
// 28672 x 8192 in groups of 64 37.5 us, 3.4 TB/s (50 %, 36 %).  Loads alone reach
// 6 TB/s, with unpacking 5.7, with the products of 8 rows 5.3 and of 16 rows 4.2.
template <int DT, int MT, int SR>
__global__ void __launch_bounds__((W4Shape<MT, SR>::THREADS), (W4Shape<MT, SR>::CTAS)) w4_kernel(const __grid_constant__ W4Args a) {
  using S = W4Shape<MT, SR>;
  extern __shared__ __align__(128) uint8_t rings[];
  __shared__ uint16_t order[FLUX_W4_MAX_ROWS];       // slots by expert
  __shared__ W4RowTile tiles[FLUX_W4_MAX_ROWS];
  int* hist = reinterpret_cast<int*>(rings);  // before the rings are used, as
  int* slot_expert = hist + FLUX_MAX_EXPERTS;
  static_assert(S::TEAMS * S::SMEM >= 4 * (FLUX_MAX_EXPERTS + FLUX_W4_MAX_ROWS), "the rings hold the routing first");
  constexpr int WARPS = S::THREADS / 32;
  __shared__ int scan[2][WARPS];
  const int thread = threadIdx.x, lane = thread & 31, cta_warp = thread >> 5;
  const int col_tiles = (a.N + W4_COLS - 1) / W4_COLS;
  wait_for_previous();
  int row_tiles;
  if (a.mode == W4_DENSE) {
    row_tiles = (a.slots + MT * 8 - 1) / (MT * 8);
    for (int i = thread; i < row_tiles; i += S::THREADS)
      tiles[i] = W4RowTile{0, static_cast<uint16_t>(i * MT * 8), static_cast<uint16_t>(min(MT * 8, a.slots - i * MT * 8))};
    for (int i = thread; i < a.slots; i += S::THREADS) order[i] = static_cast<uint16_t>(i);
    __syncthreads();
  } else {
    // stable counting sort of the slots by expert: teams that share a tile have to
    // agree on the order of its rows
    for (int e = thread; e < a.E; e += S::THREADS) hist[e] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = thread; i < a.slots; i += S::THREADS) {
      int e = a.ids[i];
      if (e >= 0 && e < a.E) {
        atomicAdd(&hist[e], 1);
      } else {
        bad = true;
        e = -1;
      }
      slot_expert[i] = e;
    }
    if (bad) atomicCAS(a.hdr, 0u, static_cast<uint32_t>(FLUX_ERR_INVALID_ARG));
    __syncthreads();
    // exclusive sums of slots and row tiles over the experts
    constexpr int PER = (FLUX_MAX_EXPERTS + S::THREADS - 1) / S::THREADS;
    int slots = 0, rt = 0;
    for (int k = 0; k < PER; ++k) {
      const int e = thread * PER + k, n = e < a.E ? hist[e] : 0;
      slots += n;
      rt += (n + MT * 8 - 1) / (MT * 8);
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
      scan[0][cta_warp] = s0;
      scan[1][cta_warp] = r0;
    }
    __syncthreads();
    s0 -= slots;
    r0 -= rt;
    row_tiles = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < cta_warp) {
        s0 += scan[0][w];
        r0 += scan[1][w];
      }
      row_tiles += scan[1][w];
    }
    for (int k = 0; k < PER; ++k) {
      const int e = thread * PER + k, n = e < a.E ? hist[e] : 0;
      if (e < a.E) hist[e] = s0;
      for (int m = 0; m < n; m += MT * 8)
        tiles[r0++] = W4RowTile{static_cast<uint16_t>(e), static_cast<uint16_t>(s0 + m),
                                static_cast<uint16_t>(min(MT * 8, n - m))};
      s0 += n;
    }
    __syncthreads();
    if (cta_warp == 0) {
      for (int i0 = 0; i0 < a.slots; i0 += 32) {
        const int i = i0 + lane, e = i < a.slots ? slot_expert[i] : -1;
        const bool in = e >= 0;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, in ? e : -1 - lane);
        const int at = in ? hist[e] : 0;
        __syncwarp();
        const int place = at + __popc(same & ((1u << lane) - 1u));
        if (in) {
          order[place] = static_cast<uint16_t>(i);
          if (lane == __ffs(same) - 1) hist[e] = at + __popc(same);
        }
        __syncwarp();
        if (blockIdx.x == 0 && i < a.slots && !in) a.where[i] = W4Slot{W4_NONE, 0};
      }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
      for (int r = cta_warp; r < row_tiles; r += WARPS)
        for (int m = lane; m < tiles[r].rows; m += 32)
          a.where[order[tiles[r].first + m]] = W4Slot{static_cast<uint16_t>(r), static_cast<uint16_t>(m)};
    }
  }

  // a team: one warp of each of the four schedulers, each of another age there
  const int warp = cta_warp % W4_WARPS, team = (cta_warp / W4_WARPS + warp) % S::TEAMS, tid = warp * 32 + lane,
            g = lane >> 2, c = lane & 3;
  uint8_t* const ring = rings + team * S::SMEM;
  const int units = row_tiles * col_tiles * a.runs;
  // every team that works has a unit
  const int teams = min(a.teams, units), me = team * gridDim.x + blockIdx.x;
  if (me >= teams) return;
  const W4Split split{units / teams, units % teams};
  if (me == 0 && tid == 0 && a.mode != W4_DENSE) *a.split = split;
  const int u0 = split.first(me), n_units = split.first(me + 1) - u0;
  int tile = u0 / a.runs, run = u0 - tile * a.runs;

  const uint32_t ring_at = smem_u32(ring), x_from = g * 256 + c * 16 + ((g & 1) << 6),
                 sc_from = S::CHUNK * S::XRUN + (warp * 16 * W4_CA + g * 4) * 2;
  constexpr int P = S::AHEAD;

  // rows of x and scales of n runs from `first` of a tile, into one buffer
  auto stage = [&](uint8_t* to, int of_tile, int first, int n) {
    const int rt_i = of_tile / col_tiles, col0 = (of_tile - rt_i * col_tiles) * W4_COLS;
    const W4RowTile rt = tiles[rt_i];
    // rows in 16-byte chunks (8 inputs): chunk 4 j + c of a row lies at
    // 4 (j ^ (row & 1)) + c, so that two rows' reads meet different banks
    const int k = tid & 15, k0 = first * W4_RUN + k * 8;
    static_assert(W4_THREADS / 16 == 8, "eight rows of x at a time");
#pragma unroll
    for (int p = 0; p < MT; ++p) {
      const int m = p * 8 + (tid >> 4);
      if (m < rt.rows) {
        const int slot = order[rt.first + m];
        const uint16_t* row = a.x + static_cast<size_t>(a.mode == W4_LAYER0 ? slot / a.topk : slot) * a.K;
        uint8_t* at = to + m * 256 + ((k ^ ((m & 1) << 2)) << 4);
        for (int r = 0; r < n; ++r) {
          const int in = k0 + r * W4_RUN;
          copy16_or_zero(at + r * S::XRUN, row + (in < a.K ? in : 0), in < a.K);
        }
      }
    }
    constexpr int AT_ONCE = W4_THREADS / (SR * W4_COLS / 8);
    const int sr = tid / (W4_COLS / 8) % SR, col = tid % (W4_COLS / 8) * 8;
    for (int r = tid / (SR * W4_COLS / 8); r < n; r += AT_ONCE) {
      const int at = (first + r) * W4_RUN + sr * (W4_RUN / SR);
      const bool in = at < a.K && col0 + col < a.N;
      const size_t from = (static_cast<size_t>(rt.expert) * a.groups + (in ? at / a.group : 0)) * a.N + (in ? col0 + col : 0);
      copy16_or_zero(to + S::CHUNK * S::XRUN + r * S::SRUN + (sr * W4_COLS + col) * 2, a.scales + from, in);
    }
  };
  // this thread's words: columns 4 g + h of the warp's 32, which are the rows g and
  // g + 8 of its two A operands; its scales and its sums are of neighbours then
  constexpr int HALVES = 2 * W4_CA;
  static_assert(HALVES == 4, "a thread's columns are four neighbours");
  const uint4* q[HALVES];
  uint4 words[P][HALVES];
  auto load_words = [&](int of_tile, int first, int n) {
    const int rt_i = of_tile / col_tiles, col = (of_tile - rt_i * col_tiles) * W4_COLS + warp * 16 * W4_CA + g * 4;
    const size_t col0 = static_cast<size_t>(tiles[rt_i].expert) * a.N;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      q[h] = reinterpret_cast<const uint4*>(a.q + ((col0 + min(col + h, a.N - 1)) * a.runs + first) * W4_RUN_BYTES + c * 16);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < n) words[i][h] = load_codes(q[h] + i * 4);
    }
  };

  int todo = n_units, buffer = 0;
  int n_runs = min(a.runs - run, todo);
  load_words(tile, run, n_runs);
  stage(ring, tile, run, min(S::CHUNK, n_runs));
  copy_commit();
#pragma unroll 1
  for (bool first_tile = true; todo > 0; first_tile = false) {
    const bool whole = n_runs == a.runs;
    todo -= n_runs;
    const int rt_i = tile / col_tiles, ct = tile - rt_i * col_tiles;
    const W4RowTile rt = tiles[rt_i];
    const int next_runs = min(a.runs, todo);  // of the next tile
    f32x2 acc[HALVES][MT] = {};  // column 4 g + h of the warp's 32, rows 2 c and 2 c + 1 of each eight
    // n runs of the tile from r0, their rows of x and scales at `at`
    auto multiply = [&](auto live_tiles, uint32_t at, int r0, int n) {
      constexpr int LIVE = decltype(live_tiles)::value;
      uint32_t x0 = at + x_from, x1 = x0 ^ 64, sc = at + sc_from;
#pragma unroll 1
      for (int r = 0; r < n; r += P) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (r + i >= n) break;
          uint32_t w[HALVES][4];
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            w[h][0] = words[i][h].x, w[h][1] = words[i][h].y, w[h][2] = words[i][h].z, w[h][3] = words[i][h].w;
            if (r0 + r + i + P < n_runs) words[i][h] = load_codes(q[h] + (i + P) * 4);
          }
          float part[W4_CA][LIVE][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 xv[LIVE];
#pragma unroll
            for (int m = 0; m < LIVE; ++m) xv[m] = shared16((j & 1 ? x1 : x0) + i * S::XRUN + (j >> 1) * 128 + m * 2048);
#pragma unroll
            for (int ca = 0; ca < W4_CA; ++ca) {
              uint32_t pa[4], pb[4];
              codes8<DT>(w[2 * ca][j], pa);
              codes8<DT>(w[2 * ca + 1][j], pb);
#pragma unroll
              for (int m = 0; m < LIVE; ++m) {
                if (j % (4 / SR) == 0) mma_16x8x16<DT, true>(part[ca][m], pa[0], pb[0], pa[1], pb[1], xv[m].x, xv[m].y);
                else mma_16x8x16<DT, false>(part[ca][m], pa[0], pb[0], pa[1], pb[1], xv[m].x, xv[m].y);
                mma_16x8x16<DT, false>(part[ca][m], pa[2], pb[2], pa[3], pb[3], xv[m].z, xv[m].w);
              }
            }
            if ((j + 1) % (4 / SR) == 0) {
              const uint32_t s = sc + i * S::SRUN + j / (4 / SR) * (W4_COLS * 2);
              f32x2 f[HALVES];
              shared_scales<DT>(s, f);
#pragma unroll
              for (int h = 0; h < HALVES; ++h)
#pragma unroll
                for (int m = 0; m < LIVE; ++m)
                  acc[h][m] = fma2(f[h], pair(part[h / 2][m][h % 2 * 2], part[h / 2][m][h % 2 * 2 + 1]), acc[h][m]);
            }
          }
        }
        x0 += P * S::XRUN;
        x1 += P * S::XRUN;
        sc += P * S::SRUN;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) q[h] += P * 4;
      }
    };
#pragma unroll 1
    for (int r0 = 0; r0 < n_runs; r0 += S::CHUNK) {
      const int n = min(S::CHUNK, n_runs - r0);
      copy_wait<0>();
      team_sync<W4_WARPS>(team);  // this buffer is filled, the other one has been read
      if (r0 + n < n_runs) stage(ring + (buffer ^ 1) * S::BUFFER, tile, run + r0 + n, min(S::CHUNK, n_runs - r0 - n));
      else if (next_runs > 0) stage(ring + (buffer ^ 1) * S::BUFFER, tile + 1, 0, min(S::CHUNK, next_runs));
      copy_commit();
      const uint32_t at = ring_at + buffer * S::BUFFER;
      buffer ^= 1;
      // by the row tiles of 8 that are there, tested here: instructions on absent
      // ones would run all the same inside the loop
      if constexpr (MT == 1) {
        multiply(std::integral_constant<int, 1>{}, at, r0, n);
      } else {
        if (rt.rows <= 8) multiply(std::integral_constant<int, 1>{}, at, r0, n);
        else if (MT == 2 || rt.rows <= 16) multiply(std::integral_constant<int, 2>{}, at, r0, n);
        else multiply(std::integral_constant<int, MT>{}, at, r0, n);
      }
    }
    ++tile;
    run = 0;
    n_runs = next_runs;
    if (next_runs > 0) load_words(tile, 0, next_runs);  // on their way while this tile is written

    // a cut tile's sums go to the workspace, by rows
    float* part = a.parts + static_cast<size_t>(2 * me + (first_tile ? 0 : 1)) * S::PART;
    const int col = warp * 16 * W4_CA + g * 4, n = ct * W4_COLS + col;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = m * 8 + 2 * c + b;
        if (r >= rt.rows || n >= a.N) continue;
        float f[HALVES];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) f[h] = b == 0 ? halves(acc[h][m]).x : halves(acc[h][m]).y;
        const float4 v = make_float4(f[0], f[1], f[2], f[3]);
        if (!whole) {
          *reinterpret_cast<float4*>(part + r * W4_COLS + col) = v;
        } else {
          const size_t at = static_cast<size_t>(order[rt.first + r]) * a.N + n;
          if (a.mode == W4_LAYER1) *reinterpret_cast<float4*>(a.rows_f32 + at) = v;
          else *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack2<DT>(v.x, v.y), pack2<DT>(v.z, v.w));
        }
      }
    }
  }
}

constexpr int W4_JOIN_WARPS = 8;

// Sums of one slot's columns n .. n + 3 in the workspace, left zero there.
template <int MT>
struct W4Parts {
  static constexpr int PART = W4_COLS * MT * 8;
  const W4Args& a;
  W4Split split;
  int col_tiles, ct, col;
  int unit, row, c0, c1;  // of the slot

  // whether several teams have sums of the slot's tile
  __device__ __forceinline__ bool open(W4Slot at) {
    unit = (at.tile * col_tiles + ct) * a.runs;
    row = at.row;
    c0 = split.team_of(unit);
    c1 = split.team_of(unit + a.runs - 1);
    return c0 != c1;
  }
  __device__ __forceinline__ float4* part(int k) const {
    // the tile is the first of team k unless it begins inside its stretch
    return reinterpret_cast<float4*>(a.parts + static_cast<size_t>(2 * k + (split.first(k) >= unit ? 0 : 1)) * PART + row * W4_COLS + col);
  }
  // adds the parts of the teams from `first` on, BATCH loads in flight together
  template <int BATCH>
  __device__ __forceinline__ void add(int first, float4& v) const {
    for (int k0 = first; k0 <= c1; k0 += BATCH) {
      float4 f[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) f[b] = *part(min(k0 + b, c1));
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (k0 + b > c1) break;
        *part(k0 + b) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        v.x += f[b].x;
        v.y += f[b].y;
        v.z += f[b].z;
        v.w += f[b].w;
      }
    }
  }
};

// The second half of a product: adds the parts of cut tiles in team order, for
// layer1 the tokens' slots, and writes zeros for slots of no expert.  Four
// columns of one row of the output per thread; layer1: a warp for each of up to
// W4_JOIN_WARPS slots of the token at a time, which meet in shared memory and are
// added in slot order (slots one after the other in one thread took twice the
// time).  Leaves what it reads of the
// workspace zero.  A chain of latencies: 8192 columns of 13 rows 5 us with cold
// caches, 4096 of 24 rows and 6 slots 8 us behind the products.
template <int DT, int MT, bool LAYER1>
__global__ void __launch_bounds__(W4_JOIN_WARPS * 32) w4_join_kernel(const __grid_constant__ W4Args a) {
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int n = (LAYER1 ? blockIdx.x * 32 + lane : blockIdx.x * blockDim.x + threadIdx.x) * 4, row = blockIdx.y;
  const int col_tiles = (a.N + W4_COLS - 1) / W4_COLS, ct = n / W4_COLS;
  W4Parts<MT> p{a, a.mode == W4_DENSE ? a.dense_split : *a.split, col_tiles, ct, n - ct * W4_COLS, 0, 0, 0, 0};
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float4 sum = zero;
  bool write = n < a.N;
  if constexpr (LAYER1) {
    __shared__ float4 meet[W4_JOIN_WARPS][32];
    for (int j0 = 0; j0 < a.topk; j0 += warps) {
      const int j = j0 + warp;
      float4 f = zero;
      if (j < a.topk && write) {
        const int slot = row * a.topk + j;
        const W4Slot at = a.where[slot];
        const float w = a.weights[slot];
        if (at.tile != W4_NONE) {
          if (p.open(at)) {
            p.template add<4>(p.c0, f);
          } else {
            float4* from = reinterpret_cast<float4*>(a.rows_f32 + static_cast<size_t>(slot) * a.N + n);
            f = *from;
            *from = zero;
          }
          f = make_float4(__fmul_rn(w, f.x), __fmul_rn(w, f.y), __fmul_rn(w, f.z), __fmul_rn(w, f.w));
        }
      }
      if (j0 > 0) __syncthreads();  // the slots before have been added
      meet[warp][lane] = f;
      __syncthreads();
      if (warp == 0) {
        sum.x += f.x;
        sum.y += f.y;
        sum.z += f.z;
        sum.w += f.w;
        for (int w = 1; w < min(warps, a.topk - j0); ++w) {
          const float4 o = meet[w][lane];
          sum.x += o.x;
          sum.y += o.y;
          sum.z += o.z;
          sum.w += o.w;
        }
      }
    }
    write = write && warp == 0;
  } else if (write) {
    const W4Slot at = a.mode == W4_DENSE ? W4Slot{static_cast<uint16_t>(row / (MT * 8)), static_cast<uint16_t>(row % (MT * 8))}
                                         : a.where[row];
    if (at.tile != W4_NONE) {
      write = p.open(at);  // else written already
      if (write) p.template add<12>(p.c0, sum);
    }
  }
  if (write)
    *reinterpret_cast<uint2*>(a.out + static_cast<size_t>(row) * a.N + n) = make_uint2(pack2<DT>(sum.x, sum.y), pack2<DT>(sum.z, sum.w));
  if (a.mode == W4_DENSE) return;
  // the last block takes the routing out of the workspace
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.joined, 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (last == 0) return;
  for (int i = threadIdx.x; i < a.slots; i += blockDim.x) a.where[i] = W4Slot{0, 0};
  if (threadIdx.x == 0) {
    *a.split = W4Split{0, 0};
    *a.joined = 0u;
  }
}

// One thread per four columns and group: the group's largest magnitude / 7,
// rounded to 16 bits, is its scale; codes are the nearest multiples of it.  Eight
// loads of 8 bytes are on their way together; the second reading of a group comes
// from L1 or L2.  Run once per weight; its stores are words 64 bytes of a column
// apart, which fill 4 bytes of a sector each: 8 x 4096 x 14336 in groups of 128
// 571 us, 2.1 TB/s; a column a thread took 844.
constexpr int W4_QUANT_COLS = 4;

template <int DT>
__global__ void __launch_bounds__(128)
w4_quantize_kernel(int K, int N, int runs, int group, int groups, const uint16_t* w, uint8_t* q,
                   uint16_t* scales) {
  constexpr int C = W4_QUANT_COLS;
  const int n = (blockIdx.x * 128 + threadIdx.x) * C;
  const size_t e = blockIdx.z;
  if (n >= N) return;
  // eight inputs of the four columns
  auto load8 = [&](int k, float (&v)[8][C]) {
    const uint16_t* from = w + (e * K + k) * N + n;
    uint2 raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = load_global(reinterpret_cast<const uint2*>(from + static_cast<size_t>(i) * N));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 lo = unpack2<DT>(raw[i].x), hi = unpack2<DT>(raw[i].y);
      v[i][0] = lo.x, v[i][1] = lo.y, v[i][2] = hi.x, v[i][3] = hi.y;
    }
  };
  for (int g = blockIdx.y; g < groups; g += gridDim.y) {
    const int k0 = g * group, k1 = K - k0 > group ? k0 + group : K;
    float top[C] = {}, v[8][C];
    for (int k = k0; k < k1; k += 8) {
      load8(k, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c) top[c] = fmaxf(top[c], fabsf(v[i][c]));
    }
    const uint32_t s01 = pack2<DT>(top[0] / 7.0f, top[1] / 7.0f), s23 = pack2<DT>(top[2] / 7.0f, top[3] / 7.0f);
    *reinterpret_cast<uint2*>(scales + (e * groups + g) * N + n) = make_uint2(s01, s23);
    const float scale[C] = {unpack2<DT>(s01).x, unpack2<DT>(s01).y, unpack2<DT>(s23).x, unpack2<DT>(s23).y};
    // the last group also fills its run of 128 inputs
    const int kend = g == groups - 1 ? runs * W4_RUN : k1;
    for (int k = k0; k < kend; k += 8) {
      uint32_t word[C] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
      if (k < K) {
        load8(k, v);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (!(scale[c] > 0.0f)) continue;
          word[c] = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int code = min(max(static_cast<int>(rintf(v[i][c] / scale[c])) + 8, 0), 15);
            word[c] |= static_cast<uint32_t>(code) << (i / 2 * 4 + i % 2 * 16);
          }
        }
      }
      const int r = k % W4_RUN;
#pragma unroll
      for (int c = 0; c < C; ++c)
        *reinterpret_cast<uint32_t*>(q + ((e * N + n + c) * runs + k / W4_RUN) * W4_RUN_BYTES + r % 32 / 8 * 16 + r / 32 * 4) =
            word[c];
    }
  }
}

// Workspace: header, how the units were cut, the slots' tiles, sums of cut tiles, fp32
// rows (used by layer1; the size is the same for all three products).
struct W4Ws {
  size_t split, where, parts, rows, total;
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
  w.split = take(sizeof(W4Split));
  w.where = take(sizeof(W4Slot) * slots);
  w.parts = take(sizeof(float) * 2 * W4_MAX_TEAMS * W4_COLS * 8 * w4_row_tiles_of_8(slots));
  w.rows = take(sizeof(float) * slots * static_cast<size_t>(N));
  w.total = at;
  return w;
}

template <int DT, int MT, int SR>
flux_status_t w4_launch(W4Args a, const DeviceInfo& dev, cudaStream_t s) {
  using S = W4Shape<MT, SR>;
  constexpr int smem = S::TEAMS * S::SMEM;
  static OncePerDevice once;
  const cudaError_t attr = once(dev.device, [] {
    return cudaFuncSetAttribute(w4_kernel<DT, MT, SR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr != cudaSuccess) return cuda_fail(attr);
  // no more teams than units (of as many row tiles as the slots can make)
  const long long col_tiles = (a.N + W4_COLS - 1) / W4_COLS;
  const long long row_tiles = a.mode == W4_DENSE ? (a.slots + MT * 8 - 1) / (MT * 8) : a.slots;
  const long long units = row_tiles * col_tiles * a.runs;
  if (units > INT_MAX) return FLUX_ERR_UNSUPPORTED;
  const long long sms = std::min(dev.sm_count, W4_MAX_TEAMS / 4), ctas = S::CTAS * sms, fill = S::TEAMS * ctas;
  a.teams = static_cast<int>(std::min(units, std::max(std::min(fill, units / W4_MIN_UNITS), sms)));
  a.dense_split = W4Split{static_cast<int>(units / a.teams), static_cast<int>(units % a.teams)};
  cudaError_t e = launch_behind(w4_kernel<DT, MT, SR>, dim3(std::min<long long>(a.teams, ctas)), S::THREADS, smem, s, a);
  if (e != cudaSuccess) return cuda_fail(e);
  // no tile is cut if the teams' stretches are whole tiles
  if (a.mode == W4_DENSE && units % a.teams == 0 && units / a.teams % a.runs == 0) return FLUX_OK;
  const int join_warps = a.mode == W4_LAYER1 ? std::min(a.topk, W4_JOIN_WARPS) : 4;
  const int join_cols = a.mode == W4_LAYER1 ? 128 : join_warps * 128;
  e = launch_behind(a.mode == W4_LAYER1 ? w4_join_kernel<DT, MT, true> : w4_join_kernel<DT, MT, false>,
                    dim3((a.N + join_cols - 1) / join_cols, a.mode == W4_LAYER1 ? a.T : a.slots), join_warps * 32, 0, s, a);
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
  // rows of one tile: all of them, and for the experts about twice what one gets
  // on the average (an expert with more rows has several tiles, whose codes
  // come from L2 again)
  const int mt = w4_row_tiles_of_8(a.mode == W4_DENSE ? a.slots : std::min(a.T, 2 * ((a.slots + a.E - 1) / a.E)));
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
  if (N % 8 != 0 || K % 8 != 0 || N > W4_MAX_SIZE || K > W4_MAX_SIZE || group % 32 != 0) return FLUX_ERR_UNSUPPORTED;
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
  a.split = reinterpret_cast<W4Split*>(ws + w.split);
  a.joined = static_cast<uint32_t*>(workspace) + WS_JOINED;
  a.where = reinterpret_cast<W4Slot*>(ws + w.where);
  a.parts = reinterpret_cast<float*>(ws + w.parts);
  a.rows_f32 = reinterpret_cast<float*>(ws + w.rows);
  a.slots = slots;
  a.T = T;
  a.N = N;
  a.K = K;
  a.runs = (K + W4_RUN - 1) / W4_RUN;
  a.group = group;
  a.groups = ceil_div(K, group);
  a.E = E;
  a.topk = topk;
  a.mode = mode;
  return dtype == FLUX_BF16 ? w4_launch_rows<1>(a, dev, s) : w4_launch_rows<0>(a, dev, s);
}

}  // namespace
}  // namespace flux

using namespace flux;

extern "C" size_t flux_w4_weight_bytes(int E, int K, int N) {
  if (E < 1 || K < 0 || N < 0 || K > W4_MAX_SIZE || N > W4_MAX_SIZE) return 0;
  return static_cast<size_t>(E) * N * ((K + W4_RUN - 1) / W4_RUN) * (W4_RUN / 2);
}

extern "C" size_t flux_w4_workspace_size(int rows, int N, int K, int E) {
  if (rows < 0 || rows > FLUX_W4_MAX_ROWS || N < 0 || K < 0 || N > W4_MAX_SIZE || K > W4_MAX_SIZE || E < 1 ||
      E > FLUX_MAX_EXPERTS)
    return 0;
  return w4_ws(rows, N).total;
}

extern "C" flux_status_t flux_w4_quantize(int E, int K, int N, int group, flux_dtype_t dtype, const void* w, void* q,
                                          void* scales, void* stream) {
  if (!w4_common_ok(N, K, group, E, dtype)) return FLUX_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0 || N > W4_MAX_SIZE || K > W4_MAX_SIZE || group % 32 != 0) return FLUX_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return FLUX_OK;
  if (w == nullptr || q == nullptr || scales == nullptr) return FLUX_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(q) || !aligned16(scales)) return FLUX_ERR_UNSUPPORTED;
  DeviceInfo dev;
  flux_status_t st = current_device(&dev);
  if (st != FLUX_OK) return st;
  const int runs = (K + W4_RUN - 1) / W4_RUN, groups = ceil_div(K, group);
  const int cols = 128 * W4_QUANT_COLS;
  const dim3 grid((N + cols - 1) / cols, std::min(groups, 65535), E);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FLUX_BF16)
    w4_quantize_kernel<1><<<grid, 128, 0, s>>>(K, N, runs, group, groups, static_cast<const uint16_t*>(w),
                                               static_cast<uint8_t*>(q), static_cast<uint16_t*>(scales));
  else
    w4_quantize_kernel<0><<<grid, 128, 0, s>>>(K, N, runs, group, groups, static_cast<const uint16_t*>(w),
                                               static_cast<uint8_t*>(q), static_cast<uint16_t*>(scales));
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
