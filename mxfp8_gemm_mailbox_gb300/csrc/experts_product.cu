// Products grouped by expert in microscaled formats, for sm_103a:
//
//   y[r][n] = sum_k W[e][n][k] x[r][k],   begin[e] <= r < begin[e + 1]
//
// W MXFP8 or MXFP4, x MXFP8 or MXFP4, FP32 sums; the result BF16, or rounded
// to MXFP8 / MXFP4 along n.  Gated: W[e] holds n gate rows, then n up rows, and
// the result is silu(gate) up.
//
// W is the MMA's A operand (a tile of 128 of its rows), the expert's rows its B
// operand, the products kind::mxf8f6f4 with one scale a block of 32: elements of
// 4 bits lie in shared memory as 16 in 16 bytes, the latter 8 unused, which is
// how the tensor copies lay them.  A tile of a gated product takes 32 gate rows,
// their 32 up rows, 32 gate rows, 32 up rows, so a block of 32 outputs is one
// warp's lanes and its partner's.
//
// Three kernels by the rows an expert has (expert_tile, below): tiles of up to 32
// rows, bound by the stream of W (two k tiles a stage, five issuers that add up
// at the end: one issued too slowly for the memory, 57.4 us for 56.2 on the step
// below); of up to 64; and pairs of CTAs on tiles of 256 rows of W x 224, bound by
// the products.  A pair's product reads 4 KB of W and 7 KB of x in each SM for 112
// clocks' work while the copies write 7.5 KB: shared memory's rate, 128 bytes a
// clock, is what there is (a stage of 4 products took 553 clocks in place of 448),
// and over milliseconds the power limit (1.6 to 1.8 GHz).
//
// Work.  begin is read on the device, so the grid is one CTA an SM, and each
// finds its share: tiles are numbered expert by expert, tiles of rows inside
// those of W (neighbouring CTAs read the same W at the same time), and go round
// by round.  Where the call's few tiles are long, they are cut along k: the pieces
// leave FP32 partials, and the last to arrive adds them in the order of k, so
// results have the same bits every time.  The tickets that tell it are zero between
// calls.
//
// Warp roles: warp 0 copies W, and x (a pair's x: warp 1); warp 1 lays the rows'
// scales for the tensor-memory copies; warps 2-5 read the sums back; warps 6..
// issue the products.  A scale copy in the products' queue costs them 60 clocks,
// three a stage of a pair: there warp 7 fetches the scales and warps 8-11 store
// them into tensor memory from registers (375 us -> 331 at the prompt below).  One
// elected lane of a converged warp copies and issues: from a branch on the lane
// number a product took a third longer.
//
// Measured (graphs of calls with inputs and outputs of their own, past twice L2
// together; comparisons in these comments alternate up to four sets, which L2 holds
// where they are small): a token's 8 experts, N 4096, K 2048, MXFP4: 10.9 us, of
// which 5.3 are the matrices at the memory's rate and some 5 the launch's wait,
// begin's latency, the deal and the first copies; 64 rows on 36 experts, gated, N
// 2048, K 4096: 52 us, 6.2 TB/s; 4096 rows at N 7168, K 16384, MXFP8: 334 us, 2.88
// PFLOP/s (297 in the first 20 ms, before the power limit; both in 4 bits 261);
// 32768 rows on 64 experts, gated, N 2048, K 4096: 414 us, 2.66 PFLOP/s (379 at
// first); 999 rows on 7 experts, gated, N 736, K 896: 10.0 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.h"
#include "mx_format.cuh"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kTileRows = 128;  // rows of W
constexpr uint32_t kWTile = kTileRows * 128;  // in shared memory, of 128 k
constexpr uint32_t kChunk = 512;  // scales of 128 rows, 4 blocks each
constexpr int kTurnPitch = 36;    // floats of an expert row in the epilogue's turn: a quarter-warp's
                                  // 16-byte reads meet no bank twice

template <bool kPair_, int kCols_, int kTiles_, int kStages_, int kPipes_, int kSmall_, int kAtOnce_>
struct Shape {
  static constexpr bool kPair = kPair_;     // two CTAs a tile
  static constexpr int kCols = kCols_;      // expert rows of a tile
  static constexpr int kTiles = kTiles_;    // k tiles of a stage
  static constexpr int kStages = kStages_;  // of the ring
  static constexpr int kPipes = kPipes_;    // issuing warps
  static constexpr int kAtOnce = kAtOnce_;  // columns that an epilogue's warp reads together
  static constexpr int kChunks = (kCols + 127) / 128;  // scale chunks of the rows
  static constexpr int kRowsALane = (kCols + 31) / 32;
  static constexpr int kStep = kPair ? 16 : 8;  // of a product's columns
  static constexpr int kXRows = kPair ? kCols / 2 : kCols;  // rows of a copy of x: all of a CTA's,
  static constexpr int kSmall = kSmall_;                    // or where there are no more than these
  static constexpr uint32_t kXTile = kXRows * 128;
  static constexpr int kThreads = kPair ? 384 : 192 + 32 * kPipes;
  static constexpr uint32_t kAccSlot = kCols < 32 ? 32 : kCols;
  static constexpr uint32_t kAcc = 2 * kPipes * kAccSlot;
  static constexpr uint32_t kSf = 4 + 4 * kChunks;  // columns of a k tile's scales
  static constexpr uint32_t kUsed = kAcc + kStages * kTiles * kSf;
  static constexpr uint32_t kColumns = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "tensor memory");
  // Each barrier is waited on by one thread in use order.
  static_assert(kStages % kPipes == 0, "slots keep their issuers");
  static_assert(kXRows % 8 == 0 && kSmall % 8 == 0, "copies of whole swizzled groups");
  static_assert(kPair ? kPipes == 1 && kTiles == 1 : kChunks == 1, "scales");
  static_assert(kCols % kAtOnce == 0, "whole reads");
  static_assert(0x7FFFFFFF - MXFP8_MAX_EXPERT_ROWS >= kCols + MXFP8_MAX_EXPERTS, "31 bits");
  // Shared memory, from a 1024-byte boundary.
  static constexpr uint32_t kX = kStages * kTiles * kWTile;
  static constexpr uint32_t kSfa = kX + kStages * kTiles * kXTile;
  static constexpr uint32_t kSfb = kSfa + kStages * kTiles * kChunk;
  // A pair's scales come four k tiles at a time: W's chunks, then the rows' codes by k tile.
  static constexpr int kQuads = 3;
  static constexpr uint32_t kQuad = 4 * (kChunk + kRowsALane * 128);
  static constexpr uint32_t kTurns =
      kPair ? kSfa + kQuads * kQuad : kSfb + kStages * kTiles * kChunk;
  static constexpr uint32_t kTables = kTurns + 4 * kAtOnce * kTurnPitch * 4;
  static constexpr uint32_t kBars = kTables + 2 * 4 * ((MXFP8_MAX_EXPERTS + 8) / 4 * 4);
  static constexpr uint32_t kMisc = kBars + 8 * (2 * kStages + 4 + 2 * kQuads);
  static constexpr uint32_t kBytes = kMisc + 32 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
  // The allocation of tensor memory waits for whoever holds some; no CTA that in turn waits
  // for another (the projection's clusters ask for a third of an SM's shared memory) may be
  // on its SM.
  static_assert(kBytes > 233472 / 3 * 2, "an SM to itself");
};
// Few rows an expert: bound by the stream of W.  Many: by the products.
using Narrow = Shape<false, 32, 2, 5, 5, 8, 8>;
using Middle = Shape<false, 64, 2, 4, 2, 32, 16>;
using Wide = Shape<true, 224, 1, 5, 1, 56, 32>;
constexpr int kMinPiece = 16;  // k tiles of a piece of a cut tile

__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void pair_barrier(int pair) {
  asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory");
}

// To some 2^-22 of the value, subnormal ones too (to their steps).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The same, of a number in 1 .. 2.
__device__ __forceinline__ float reciprocal_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The k tiles of one tile, or a piece of them.
struct Segment {
  int expert, row, rows, w_tile;  // rows: of the tile
  int kt0, kt1;  // whole stages, but for the last of a tile
  int cut;       // which of the tiles that are cut
};

// The segments of a CTA, in order; every role walks the same list.  Tiles go round by
// round, one a CTA; with kCuts those of a round that fills half of the CTAs or less are
// cut along k into as many equal pieces as there are CTAs a tile.
template <class S, bool kCuts>
struct Share {
  const int* rows;   // [experts + 1] each expert's first row
  const int* tiles;  // [experts + 1] ... first tile
  int experts, k_tiles, stages;  // stages of a tile
  int grid, cta, round;          // in pairs where they share a tile
  int all;                       // tiles
  int rounds, pieces, piece, of; // kCuts: whole rounds; a cut tile's pieces, this CTA's piece and tile

  __device__ __forceinline__ Share(const int* r, const int* t, int e, int kt)
      : rows(r), tiles(t), experts(e), k_tiles(kt) {
    constexpr int kSharers = S::kPair ? 2 : 1;
    stages = (kt + S::kTiles - 1) / S::kTiles;
    grid = gridDim.x / kSharers;
    cta = blockIdx.x / kSharers;
    all = tiles[e];
    round = 0;
    if constexpr (kCuts) {
      rounds = static_cast<int>(static_cast<uint32_t>(all) / static_cast<uint32_t>(grid));
      const int left = all - rounds * grid;
      pieces = left == 0 ? 1
                         : max(1, min(static_cast<int>(static_cast<uint32_t>(grid) /
                                                       static_cast<uint32_t>(left)),
                                      stages * S::kTiles / kMinPiece));
      of = static_cast<int>(static_cast<uint32_t>(cta) / static_cast<uint32_t>(pieces));
      piece = cta - of * pieces;
    }
  }
  __device__ __forceinline__ bool next(Segment& s) {
    int tile = cta + grid * round;
    s.kt0 = 0;
    s.kt1 = k_tiles;
    if constexpr (kCuts) {
      s.cut = of;
      if (round == rounds) {
        tile = rounds * grid + of;
        s.kt0 = piece * stages / pieces * S::kTiles;
        s.kt1 = min(k_tiles, (piece + 1) * stages / pieces * S::kTiles);
      } else if (round > rounds) {
        return false;
      }
    }
    ++round;
    if (tile >= all) return false;
    // The last expert whose first tile is not past this one: eight at a time, whose loads
    // do not wait for one another.
    int lo = 0;
    static_assert(MXFP8_MAX_EXPERTS <= 512, "three steps of eight");
#pragma unroll
    for (int step = 64; step > 0; step /= 8) {
      if (step >= experts) continue;
      int past = 0;
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const int e = lo + i * step;
        past += e < experts && tiles[min(e, experts)] <= tile;
      }
      lo += past * step;
    }
    s.expert = lo;
    const uint32_t count = rows[lo + 1] - rows[lo];
    const uint32_t row_tiles = (count + S::kCols - 1) / S::kCols;
    const uint32_t local = tile - tiles[lo];
    s.w_tile = local;
    int first = 0, size = count;
    if (row_tiles > 1) {  // equal tiles of rows, in whole steps of a product
      s.w_tile = local / row_tiles;
      size = ((count + row_tiles - 1) / row_tiles + S::kStep - 1) / S::kStep * S::kStep;
      first = (local - s.w_tile * row_tiles) * size;
    }
    s.row = rows[lo] + first;
    s.rows = min(size, static_cast<int>(count) - first);
    return true;
  }
  __device__ __forceinline__ uint32_t count(const Segment& s) const {  // stages
    return static_cast<uint32_t>((s.kt1 - s.kt0 + S::kTiles - 1) / S::kTiles);
  }
};

// The experts' first rows and first tiles.  Rows outside 0 .. rows or that go back are
// cut and raise the flag.  All threads load (one latency), one warp adds, a run of
// consecutive experts a lane.
__device__ __forceinline__ void deal(const ExpertParams& p, int cols, int w_tiles, int* rows,
                                     int* tiles) {
  bool bad = false;
  for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) {
    const int given = p.begin ? p.begin[e] : e * p.rows;  // without begin: one expert
    const int b = min(max(given, 0), p.rows);
    bad |= given != b;
    rows[e] = b;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (p.experts + 32) / 32;
    const int from = min(lane * per, p.experts + 1), to = min(from + per, p.experts + 1);
    int top = 0;
    for (int e = from; e < to; ++e) top = max(top, rows[e]);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(~0u, top, o);
      if (lane >= o) top = max(top, up);
    }
    int last = __shfl_up_sync(~0u, top, 1);  // the largest before this lane's
    if (lane == 0) last = 0;
    int sum = 0;
    const int before = last;
    for (int e = from; e < to; ++e) {
      const int b = rows[e], m = max(b, last);
      bad |= m != b;
      rows[e] = m;
      if (e > 0) sum += (m - last + cols - 1) / cols * w_tiles;
      last = m;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += up;
    }
    // tiles[e]: of the experts before e.
    int at = inc - sum;
    last = before;
    for (int e = from; e < to; ++e) {
      const int m = rows[e];
      if (e > 0) at += (m - last + cols - 1) / cols * w_tiles;
      tiles[e] = at;
      last = m;
    }
  }
  if (bad && blockIdx.x == 0 && p.flags) atomicOr(p.flags, MXFP8_FLAG_BAD_INDEX);
}

// kOut consecutive outputs from n on of one expert row to memory, where they are `live`;
// 32 / kOut neighbouring lanes have a block of 32.
template <int kOut>
__device__ __forceinline__ void store_outputs(const ExpertParams& p, const float (&v)[kOut],
                                              int row, bool live, int n) {
  if (p.format == MXFP8_FORMAT_BF16) {
    uint32_t w[kOut / 2];
#pragma unroll
    for (int i = 0; i < kOut / 2; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    uint16_t* const to = static_cast<uint16_t*>(p.out) + static_cast<size_t>(row) * p.n + n;
    if constexpr (kOut == 4) {
      if (live && n < p.n) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kOut; i += 8)
        if (live && n + i < p.n)
          ptx::st_v4(to + i, make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]));
    }
    return;
  }
  // Magnitudes as integers keep their order, and what is not finite lies above.
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < kOut; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const bool wide = p.format == MXFP8_FORMAT_MXFP8;
  bool finite = top < 0x7F800000u;
  if (wide && !finite) {  // the scale is that of the finite ones
    top = 0u;
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      if (m < 0x7F800000u) top = max(top, m);
    }
  }
#pragma unroll
  for (int o = 1; o < 32 / kOut; o *= 2) top = max(top, __shfl_xor_sync(~0u, top, o));
  live = live && n < p.n;  // n is whole blocks
  const size_t first = static_cast<size_t>(row) * p.n + n;
  uint8_t* const codes = static_cast<uint8_t*>(p.out);
  uint32_t code;
  if (wide) {
    code = scale_code(__uint_as_float(top));
    const float s = inverse_scale(code);
    uint32_t w[kOut / 4];
#pragma unroll
    for (int i = 0; i < kOut; i += 2) {
      float a = v[i] * s, b = v[i + 1] * s;
      if (!finite) {
        if (!isfinite(v[i])) a = __uint_as_float(0x7FC00000u);
        if (!isfinite(v[i + 1])) b = __uint_as_float(0x7FC00000u);
      }
      const uint32_t both = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
      w[i / 4] = i % 4 ? w[i / 4] | both << 16 : both;
    }
    if (live) {
      if constexpr (kOut == 16)
        ptx::st_v4(codes + first, make_uint4(w[0], w[1], w[2], w[3]));
      else if constexpr (kOut == 8)
        *reinterpret_cast<uint2*>(codes + first) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(codes + first) = w[0];
    }
  } else {
    finite = top < 0x7F800000u;  // of the whole block
    code = finite ? scale_code_e2m1(__uint_as_float(top)) : 255u;
    const float s = inverse_scale(code);
    uint64_t w = 0u;
#pragma unroll
    for (int i = 0; i < kOut; i += 2)
      w |= static_cast<uint64_t>(__nv_cvt_float2_to_fp4x2(make_float2(v[i] * s, v[i + 1] * s),
                                                          __NV_E2M1, cudaRoundNearest))
           << 4 * i;
    if (!finite) w = 0u;
    if (live) {
      if constexpr (kOut == 16)
        *reinterpret_cast<uint64_t*>(codes + first / 2) = w;
      else if constexpr (kOut == 8)
        *reinterpret_cast<uint32_t*>(codes + first / 2) = static_cast<uint32_t>(w);
      else
        *reinterpret_cast<uint16_t*>(codes + first / 2) = static_cast<uint16_t>(w);
    }
  }
  if (live && n % 32 == 0) p.out_scale[first / 32] = static_cast<uint8_t>(code);
}

template <class S, bool kGated, bool kCuts>
__global__ void __launch_bounds__(S::kThreads, 1)
    expert_kernel(const __grid_constant__ CUtensorMap tmap_w,
                  const __grid_constant__ CUtensorMap tmap_x,
                  const __grid_constant__ CUtensorMap tmap_x_small,
                  const __grid_constant__ ExpertParams p) {
  constexpr int kSharers = S::kPair ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  uint8_t* const smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = ptx::smem_addr(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t bar_full = sbase + S::kBars, bar_empty = bar_full + 8 * S::kStages;
  const uint32_t bar_acc_full = bar_empty + 8 * S::kStages, bar_acc_empty = bar_acc_full + 16;
  const uint32_t bar_quad_full = bar_acc_empty + 16, bar_quad_empty = bar_quad_full + 8 * S::kQuads;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  int* const rows = reinterpret_cast<int*>(smem + S::kTables);
  int* const tiles = rows + (MXFP8_MAX_EXPERTS + 8) / 4 * 4;

  // What the deal reads first, while the kernel before still runs.
  if (p.begin && tid * 32 <= p.experts) ptx::prefetch_l2_line(p.begin + tid * 32);
  const uint32_t rank = S::kPair ? ptx::cluster_ctarank() : 0;
  // At a barrier of the CTA that issues the products.
  const auto arrive = [&](uint32_t bar) {
    if constexpr (S::kPair)
      ptx::mbar_arrive_remote(ptx::map_to_rank(bar, 0));
    else
      ptx::mbar_arrive(bar);
  };

  if (tid == 0) {
    ptx::prefetch_tensormap(&tmap_w);
    ptx::prefetch_tensormap(&tmap_x);
    ptx::prefetch_tensormap(&tmap_x_small);
    for (int s = 0; s < S::kStages; ++s) {
      // The copies, and the warps of the scales.
      ptx::mbar_init(bar_full + 8 * s, S::kPair ? 2 + 2 * 4 : 2);
      ptx::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int q = 0; S::kPair && q < S::kQuads; ++q) {
      ptx::mbar_init(bar_quad_full + 8 * q, 1);
      ptx::mbar_init(bar_quad_empty + 8 * q, 4);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar_acc_full + 8 * b, S::kPipes);
      ptx::mbar_init(bar_acc_empty + 8 * b, 4 * kSharers);  // the warps that read them
    }
    ptx::fence_mbarrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 6) {
    if constexpr (S::kPair) {
      ptx::tmem_alloc_pair(sbase + S::kMisc, S::kColumns);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(sbase + S::kMisc, S::kColumns);
      ptx::tmem_relinquish();
    }
    // Not before: a CTA of the next kernel must not hold what this one waits for.
    ptx::launch_dependents();
  }
  ptx::grid_dependency_wait();
  deal(p, S::kCols, (p.w_tiles + kSharers - 1) / kSharers, rows, tiles);
  ptx::tc_fence_before();
  if constexpr (S::kPair)
    ptx::cluster_sync();  // the pair's barriers exist
  else
    __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  const auto timed_out = [&] {
    if (p.flags) atomicOr(p.flags, MXFP8_FLAG_GEMM_TIMEOUT);
  };
  Share<S, kCuts> share(rows, tiles, p.experts, p.k_tiles);
  Segment s;

  if (warp == 0 || (S::kPair && warp == 1)) {
    // ---------------------------------------------------------------- copies
    // (The warp stays converged and one elected lane copies, as in the products below.)
    {
      const bool of_w = warp == 0, of_x = !S::kPair || !of_w;
      uint32_t stage = 0;  // of all this CTA's stages; the slot's use: stage / kStages
      bool ok = true;
      while (ok && share.next(s)) {
        // A pair's CTAs have a tile of W each (the last may have none: what is copied then
        // is not stored) and half of the columns.
        const int w_tile = s.w_tile * kSharers + static_cast<int>(rank);
        const int columns = (s.rows + S::kStep - 1) / S::kStep * S::kStep / kSharers;
        const int row = s.row + static_cast<int>(rank) * columns;
        const bool small = columns <= S::kSmall;
        const uint32_t x_bytes = small ? p.x_small_bytes : p.x_bytes;
        // Gated: blocks of 32 rows are numbered through all experts' halves.
        const int w1 = kGated ? 0 : w_tile * kTileRows;
        const int w3 = kGated ? s.expert * (p.n / 16) + w_tile * 2 : s.expert;
        const uint8_t* const sf =
            p.w_sf + static_cast<size_t>(s.expert * p.w_tiles + w_tile) * p.k_tiles * kChunk;
        for (int kt = s.kt0; kt < s.kt1; kt += S::kTiles, ++stage) {
          const uint32_t slot = stage % S::kStages, use = stage / S::kStages;
          ok = __all_sync(~0u, ptx::mbar_wait(bar_empty + 8 * slot, (use & 1) ^ 1, kWaitNs));
          if (!ok) {
            timed_out();
            break;
          }
          const uint32_t full = bar_full + 8 * slot;
          const uint32_t chunks = S::kPair ? 0 : min(S::kTiles, s.kt1 - kt) * kChunk;
          if (!ptx::elect_one()) continue;
          if (rank == 0)
            ptx::mbar_arrive_expect_tx(
                full, kSharers * ((of_w ? p.w_bytes : 0) + (of_x ? x_bytes : 0)) + chunks);
          const uint32_t done = S::kPair ? ptx::map_to_rank(full, 0) : full;
          if (of_w) {
            ptx::tma_load_5d<S::kPair>(sbase + slot * S::kTiles * kWTile, &tmap_w, 0, w1, 0, w3, kt,
                                       done);
            if constexpr (!S::kPair)
              ptx::bulk_load(sbase + S::kSfa + slot * S::kTiles * kChunk,
                             sf + static_cast<size_t>(kt) * kChunk, chunks, full);
          }
          if (of_x)
            ptx::tma_load_3d<S::kPair>(sbase + S::kX + slot * S::kTiles * S::kXTile,
                                       small ? &tmap_x_small : &tmap_x,
                                       S::kTiles == 1 ? kt * 128 : 0, row,
                                       S::kTiles == 1 ? 0 : kt, done);
        }
      }
      // The products that read the last stages are done before the CTA leaves, and
      // with them the copies.
      for (int i = 0; i < S::kStages; ++i, ++stage)
        ptx::mbar_wait(bar_empty + 8 * (stage % S::kStages), ((stage / S::kStages) & 1) ^ 1,
                       kWaitNs);
    }
  } else if (S::kPair && warp == 7) {
    // ------------------------------------------------ a pair's scales, into shared memory
    uint32_t quad = 0;  // of all this CTA's; the place's use: quad / kQuads
    bool ok = true;
    while (ok && share.next(s)) {
      const int w_tile = min(s.w_tile * kSharers + static_cast<int>(rank), p.w_tiles - 1);
      const uint8_t* const of_w =
          p.w_sf + static_cast<size_t>(s.expert * p.w_tiles + w_tile) * p.k_tiles * kChunk;
      // Rows of codes on 16-byte boundaries give four k tiles a load.
      const bool wide = p.k_tiles % 4 == 0 && reinterpret_cast<uintptr_t>(p.x_scale) % 16 == 0;
      for (int kt = s.kt0; kt < s.kt1; kt += 4, ++quad) {
        const uint32_t place = quad % S::kQuads, use = quad / S::kQuads;
        const int count = min(4, s.kt1 - kt);
        uint32_t v[S::kRowsALane][4];
#pragma unroll
        for (int i = 0; i < S::kRowsALane; ++i) {
          const uint8_t* const from =
              p.x_scale +
              (static_cast<size_t>(s.row + min(lane + 32 * i, s.rows - 1)) * p.k_tiles + kt) * 4;
          if (32 * i >= s.rows) {
            v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0u;
          } else if (wide) {
            const uint4 u = *reinterpret_cast<const uint4*>(from);
            v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[i][j] = j < count ? *reinterpret_cast<const uint32_t*>(from + 4 * j) : 0u;
          }
        }
        ok = __all_sync(~0u, ptx::mbar_wait(bar_quad_empty + 8 * place, (use & 1) ^ 1, kWaitNs));
        if (!ok) {
          timed_out();
          break;
        }
        uint8_t* const to = smem + S::kSfa + place * S::kQuad;
        uint32_t* const codes = reinterpret_cast<uint32_t*>(to + 4 * kChunk);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < S::kRowsALane; ++i)
            codes[(j * S::kRowsALane + i) * 32 + lane] = v[i][j];
        __syncwarp();
        if (ptx::elect_one()) {
          const uint32_t full = bar_quad_full + 8 * place;
          ptx::mbar_arrive_expect_tx(full, count * kChunk);
          ptx::bulk_load(ptx::smem_addr(to), of_w + static_cast<size_t>(kt) * kChunk,
                         count * kChunk, full);
        }
      }
    }
    // (The last copies land before the scales' warps read them, and those before the end.)
  } else if (S::kPair && warp >= 8) {
    // ---------------- and on into tensor memory (a warp a quarter of its lanes, which all
    // hold the same)
    if constexpr (S::kPair) {
      const uint32_t lanes = static_cast<uint32_t>((warp - 8) * 32) << 16;
      uint32_t stage = 0, quad = 0;
      bool ok = true;
      while (ok && share.next(s)) {
        for (int kt = s.kt0; ok && kt < s.kt1; kt += 4, ++quad) {
          const uint32_t place = quad % S::kQuads, use = quad / S::kQuads;
          const int count = min(4, s.kt1 - kt);
          ok = __all_sync(~0u, ptx::mbar_wait(bar_quad_full + 8 * place, use & 1, kWaitNs));
          const uint8_t* const from = smem + S::kSfa + place * S::kQuad;
          const uint32_t* const codes = reinterpret_cast<const uint32_t*>(from + 4 * kChunk);
          for (int j = 0; ok && j < count; ++j, ++stage) {
            const uint4 a = *reinterpret_cast<const uint4*>(from + j * kChunk + lane * 16);
            const uint32_t ra[4] = {a.x, a.y, a.z, a.w};
            uint32_t rb[8] = {};
#pragma unroll
            for (int i = 0; i < S::kRowsALane; ++i)
              rb[i] = codes[(j * S::kRowsALane + i) * 32 + lane];
            if (j == count - 1) {
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar_quad_empty + 8 * place);
            }
            const uint32_t slot = stage % S::kStages;
            ok = __all_sync(~0u, ptx::mbar_wait(bar_empty + 8 * slot,
                                                (stage / S::kStages & 1) ^ 1, kWaitNs));
            const uint32_t to = tmem + lanes + S::kAcc + slot * S::kSf;
            ptx::tc_fence_after();
            ptx::tmem_st_32x32b_x4(to, ra);
            ptx::tmem_st_32x32b_x8(to + 4, rb);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar_full + 8 * slot);
          }
          if (!ok) timed_out();
        }
      }
    }
  } else if (!S::kPair && warp == 1) {
    // ------------------------------------------- the rows' scales, laid for the copy
    // Row r's four codes of a k tile at (r % 32) 16 + (r / 32) 4 of its chunk.  Four k
    // tiles' loads are under way while the four before are stored.
    constexpr int kAhead = 4;
    static_assert(kAhead % S::kTiles == 0, "whole stages");
    uint32_t stage = 0;
    bool ok = true;
    while (ok && share.next(s)) {
      const uint8_t* at[S::kRowsALane];
#pragma unroll
      for (int i = 0; i < S::kRowsALane; ++i)
        at[i] = p.x_scale +
                static_cast<size_t>(s.row + min(lane + 32 * i, s.rows - 1)) * p.k_tiles * 4;
      uint32_t next[kAhead][S::kRowsALane];
      const auto load = [&](int kt) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int i = 0; i < S::kRowsALane; ++i)
            next[j][i] = kt + j < s.kt1 && 32 * i < s.rows
                             ? *reinterpret_cast<const uint32_t*>(at[i] + 4 * (kt + j))
                             : 0u;
      };
      load(s.kt0);
      for (int kt = s.kt0; ok && kt < s.kt1; kt += kAhead) {
        uint32_t now[kAhead][S::kRowsALane];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int i = 0; i < S::kRowsALane; ++i) now[j][i] = next[j][i];
        load(kt + kAhead);
#pragma unroll
        for (int j0 = 0; j0 < kAhead; j0 += S::kTiles) {
          if (kt + j0 >= s.kt1) break;
          const uint32_t slot = stage % S::kStages, use = stage / S::kStages;
          ok = __all_sync(~0u, ptx::mbar_wait(bar_empty + 8 * slot, (use & 1) ^ 1, kWaitNs));
          if (!ok) {
            timed_out();
            break;
          }
#pragma unroll
          for (int j = 0; j < S::kTiles; ++j)
#pragma unroll
            for (int i = 0; i < S::kRowsALane; ++i)
              *reinterpret_cast<uint32_t*>(smem + S::kSfb + (slot * S::kTiles + j) * kChunk +
                                           lane * 16 + i * 4) = now[j0 + j][i];
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive(bar_full + 8 * slot);
          ++stage;
        }
      }
    }
  } else if (warp >= 6) {
    // -------------------------------------------------------------- products
    // The warp stays converged and one elected lane issues: issued from a branch on the lane
    // number a product took about a third longer.
    if (rank == 0) {
      const uint32_t pipe = warp - 6;
      uint32_t stage = pipe, before = 0, use = 0;  // use: segments so far
      bool ok = true;
      const auto commit = [&](uint32_t bar) {
        if constexpr (S::kPair)
          ptx::mma_commit_pair(bar);
        else
          ptx::mma_commit(bar);
      };
      while (ok && share.next(s)) {
        const uint32_t count = share.count(s), buffer = use & 1;
        const uint32_t columns =
            static_cast<uint32_t>((s.rows + S::kStep - 1) / S::kStep * S::kStep);
        const uint32_t idesc = p.idesc | columns >> 3 << 17;
        const uint32_t x_tile = (columns / kSharers <= S::kSmall ? S::kSmall : S::kXRows) * 128;
        const uint32_t acc = tmem + (buffer * S::kPipes + pipe) * S::kAccSlot;
        ok = __all_sync(~0u,
                        ptx::mbar_wait(bar_acc_empty + 8 * buffer, ((use >> 1) & 1) ^ 1, kWaitNs));
        if (!ok) {
          timed_out();
          break;
        }
        ptx::tc_fence_after();
        uint32_t more = 0u;  // onto the sums of the stages before
        for (; stage < before + count; stage += S::kPipes) {
          const uint32_t slot = stage % S::kStages;
          ok = __all_sync(~0u,
                          ptx::mbar_wait(bar_full + 8 * slot, (stage / S::kStages) & 1, kWaitNs));
          if (!ok) {
            timed_out();
            break;
          }
          ptx::tc_fence_after();
          const int left = s.kt1 - s.kt0 - static_cast<int>(stage - before) * S::kTiles;
          if (ptx::elect_one()) {
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t) {
              if (t >= left) break;
              const uint32_t tile = slot * S::kTiles + t;
              const uint32_t sfa = tmem + S::kAcc + tile * S::kSf, sfb = sfa + 4;
              if constexpr (!S::kPair) {
                ptx::tmem_cp_32x128b_warpx4(sfa, ptx::desc_rows16(sbase + S::kSfa + tile * kChunk));
                ptx::tmem_cp_32x128b_warpx4(sfb, ptx::desc_rows16(sbase + S::kSfb + tile * kChunk));
              }
              const uint32_t a = sbase + tile * kWTile;
              const uint32_t b = sbase + S::kX + slot * S::kTiles * S::kXTile + t * x_tile;
#pragma unroll
              for (uint32_t kb = 0; kb < 4; ++kb) {
                const uint64_t ad = ptx::desc_kmajor_sw128(a + 32 * kb);
                const uint64_t bd = ptx::desc_kmajor_sw128(b + 32 * kb);
                if constexpr (S::kPair)
                  ptx::mma_mxf8_pair(acc, ad, bd, idesc | kb << 4 | kb << 29,
                                     t + kb > 0 ? 1u : more, sfa, sfb);
                else
                  ptx::mma_mxf8(acc, ad, bd, idesc | kb << 4 | kb << 29,
                                t + kb > 0 ? 1u : more, sfa, sfb);
              }
            }
            commit(bar_empty + 8 * slot);
          }
          __syncwarp();
          more = 1u;
        }
        before += count;
        ++use;
        if (ok && ptx::elect_one()) commit(bar_acc_full + 8 * buffer);
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp % 4;  // the tensor memory lanes this warp reaches
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr int kC = S::kAtOnce;
    // The turn: a lane has one row of W's sums of kC expert rows; it takes several outputs
    // of one expert row instead, through shared memory.  Gated: an even quarter of the
    // lanes has the gates, the odd one after it the ups, and each of their warps takes half
    // of the expert rows.
    constexpr int kRows = kGated ? kC / 2 : kC < 16 ? kC : 16;  // expert rows at a time
    constexpr int kShare = 32 / kRows;                          // lanes of one
    const int pair = quarter / 2;
    const bool gates = quarter % 2 == 0;
    float* const turns = reinterpret_cast<float*>(smem + S::kTurns);
    const int t = lane / kShare, n_lane = lane % kShare * kRows;
    // kC rows' sums of this lane's row of W.
    const auto finish = [&](const Segment& s, int c, const float (&v)[kC]) {
      float* const turn = turns + quarter * kC * kTurnPitch;
#pragma unroll
      for (int j = 0; j < kC; ++j) turn[j * kTurnPitch + lane] = v[j];
      const int w_tile = s.w_tile * kSharers + static_cast<int>(rank);
      const auto read = [&](const float* from, float (&x)[kRows]) {
#pragma unroll
        for (int i = 0; i < kRows; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(from + i);
          x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
        }
      };
      if constexpr (kGated) {
        pair_barrier(pair);
        const int at = (gates ? 0 : kRows) + t;
        const float* const mine = turn + at * kTurnPitch + n_lane;
        const int other = gates ? kC * kTurnPitch : -kC * kTurnPitch;
        float g[kRows], u[kRows];
        read(gates ? mine : mine + other, g);
        read(gates ? mine + other : mine, u);
        pair_barrier(pair);  // both have read; the next rows may come
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          // g / (1 + e^-g) u, for g < 0 as g e^g / (1 + e^g) u, with the root of the exponential
          // on both factors and the divisor, in 1 .. 2, on g alone: nothing on the way overflows
          // where the result does not (u g before the divisor did, in the last 27 % below 2^128),
          // and the root, subnormal from g = -175 on, is zero only where the result is less than
          // every format's smallest.
          const float root = exp2_approx(-0.72134752f * fabsf(g[i])), f = g[i] < 0.0f ? root : 1.0f;
          u[i] = (u[i] * f) * ((g[i] * f) * reciprocal_approx(fmaf(root, root, 1.0f)));
        }
        store_outputs<kRows>(p, u, s.row + c + at, c + at < s.rows, w_tile * 64 + pair * 32 + n_lane);
      } else {
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kC; r += kRows) {
          float x[kRows];
          read(turn + (r + t) * kTurnPitch + n_lane, x);
          store_outputs<kRows>(p, x, s.row + c + r + t, c + r + t < s.rows,
                               w_tile * kTileRows + quarter * 32 + n_lane);
        }
        __syncwarp();
      }
    };
    uint32_t before = 0, use = 0;
    bool ok = true;  // else the walk goes on without waiting: all warps meet at its barriers
    while (share.next(s)) {
      const uint32_t count = share.count(s), buffer = use & 1;
      if (ok && !ptx::mbar_wait(bar_acc_full + 8 * buffer, (use >> 1) & 1, kWaitNs)) {
        timed_out();
        ok = false;
      }
      __syncwarp();
      ptx::tc_fence_after();
      const bool whole = !kCuts || (s.kt0 == 0 && s.kt1 == p.k_tiles);
      // A piece's partials: a CTA has one cut tile at most.
      const auto place = [&](int cta) {
        return p.partial + static_cast<size_t>(cta) * kTileRows * S::kCols + quarter * 32 + lane;
      };
      for (int c = 0; c < s.rows; c += kC) {
        float v[kC];
#pragma unroll
        for (int j = 0; j < kC; ++j) v[j] = 0.0f;
        __syncwarp();  // the reads are a converged warp's
        uint32_t r[S::kPipes][kC];
#pragma unroll
        for (uint32_t q = 0; q < S::kPipes; ++q) {
          const uint32_t from = tmem + lanes + (buffer * S::kPipes + q) * S::kAccSlot + c;
          if constexpr (kC == 32)
            ptx::tmem_ld_32x32b_x32(from, r[q]);
          else if constexpr (kC == 16)
            ptx::tmem_ld_32x32b_x16(from, r[q]);
          else
            ptx::tmem_ld_32x32b_x8(from, r[q]);
        }
        ptx::tmem_wait_ld();
#pragma unroll
        for (uint32_t q = 0; q < S::kPipes; ++q) {
          if ((q + S::kPipes - before % S::kPipes) % S::kPipes >= count)
            continue;  // an issuer without a stage
#pragma unroll
          for (int j = 0; j < kC; ++j) v[j] += __uint_as_float(r[q][j]);
        }
        if (whole) {
          finish(s, c, v);
        } else {
          float* const to = place(share.cta);
#pragma unroll
          for (int j = 0; j < kC; ++j) __stcg(to + (c + j) * kTileRows, v[j]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(bar_acc_empty + 8 * buffer);
      if constexpr (kCuts) {
        if (!whole) {
          // The barrier hands the warps' partials to one thread, whose arrival releases
          // them; the last one's acquires the others' for its warps the same way.
          epilogue_barrier();
          if (tid == 64) {
            int32_t* const ticket = p.tickets + s.cut;
            misc[1] =
                ptx::atom_add_acq_rel(ticket, 1u) == static_cast<uint32_t>(share.pieces - 1);
            if (misc[1]) *ticket = 0;  // for the next call
          }
          epilogue_barrier();
          if (misc[1]) {
            for (int c = 0; c < s.rows; c += kC) {
              float v[kC];
#pragma unroll
              for (int j = 0; j < kC; ++j) v[j] = 0.0f;
              // Several pieces' loads at a time, added in the order of k.
              constexpr int kPieces = 64 / kC;
              const int lo = s.cut * share.pieces, hi = lo + share.pieces - 1;
              for (int cta = lo; cta <= hi; cta += kPieces) {
                float x[kPieces][kC];
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                  const float* const from = place(min(cta + i, hi));
#pragma unroll
                  for (int j = 0; j < kC; ++j)
                    x[i][j] = cta + i <= hi ? __ldcg(from + (c + j) * kTileRows) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
#pragma unroll
                  for (int j = 0; j < kC; ++j) v[j] += x[i][j];
              }
              finish(s, c, v);
            }
          }
        }
      }
      before += count;
      ++use;
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  if constexpr (S::kPair)
    ptx::cluster_sync();  // the pair's products read both CTAs' memories
  else
    __syncthreads();
  if (warp == 6) {
    ptx::tc_fence_after();
    if constexpr (S::kPair)
      ptx::tmem_dealloc_pair(tmem, S::kColumns);
    else
      ptx::tmem_dealloc(tmem, S::kColumns);
  }
}

// W's scales as the tensor-memory copies read them: [expert][tile][k tile], a chunk of
// 512 bytes each, lane a's four codes at (a % 32) 16 + (a / 32) 4.  Lane a of tile j holds
// row 128 j + a, or gated output 64 j + 32 (a / 64) + a % 32 of the half a / 32 % 2.
__global__ void __launch_bounds__(128) lay_scales_kernel(const uint8_t* scale, uint8_t* laid, int n,
                                                         bool gated, int w_tiles, int k_tiles) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const int a = threadIdx.x, kt = blockIdx.x, j = blockIdx.y, e = blockIdx.z;
  const int output = gated ? j * 64 + a / 64 * 32 + a % 32 : j * kTileRows + a;
  uint32_t codes = 0x7F7F7F7Fu;
  if (output < n) {
    const size_t row = static_cast<size_t>(e) * (gated ? 2 * n : n) +
                       (gated ? a / 32 % 2 * n : 0) + output;
    codes = *reinterpret_cast<const uint32_t*>(scale + (row * k_tiles + kt) * 4);
  }
  uint8_t* chunk = laid + ((static_cast<size_t>(e) * w_tiles + j) * k_tiles + kt) * kChunk;
  *reinterpret_cast<uint32_t*>(chunk + a % 32 * 16 + a / 32 * 4) = codes;
}

template <class S, bool kGated, bool kCuts>
cudaError_t launch_as(const ExpertMaps& maps, const ExpertParams& p, int ctas,
                      cudaStream_t stream) {
  const auto kernel = expert_kernel<S, kGated, kCuts>;
  static std::atomic<uint64_t> asked{0};  // a bit a device
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0u;
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(S::kBytes));
    if (e != cudaSuccess) return e;
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S::kPair ? 2 : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(S::kThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(S::kPair ? ctas / 2 * 2 : ctas));
  cfg.dynamicSmemBytes = S::kBytes;
  return cudaLaunchKernelEx(&cfg, kernel, maps.w, maps.x, maps.x_small, p);
}

}  // namespace

size_t expert_partial_bytes(int ctas) {
  return static_cast<size_t>(ctas) * kTileRows * Middle::kCols * 4;
}

// By what the host knows, the mean of an expert's rows.  A rule found on 161 shapes of 1 to
// 16384 rows, 1 to 64 experts, N and K up to 7168 x 8192, each timed as all three; its choice
// takes 1 % longer than the best on average, 17 % at the most.  Narrow, middle, wide in us:
//   8 experts x 8 rows, 2048 x 2048               6.4  6.7  8.9
//   8 experts x 24 rows, 2048 x 2048              8.6  7.2  9.1   (past 32 rows two tiles)
//   64 experts x 64 rows, 1024 x 2048            27.9 22.0 25.6
//   one expert x 64 rows, 2048 x 2048             5.6  6.0  8.2   (few tiles)
//   one expert x 256 rows, 7168 x 8192           30.8 27.2 23.2
//   22 experts x 697 rows, 112 x 128              8.0  6.5  9.5   (half of the pairs' CTAs idle)
//   9 experts x 860 rows, gated 1728 x 2688     136.2 89.1 59.0
// and cutting (by 24 k tiles saved, 40 where there are more partials), one matrix,
// whole and cut, at 1 row and K = 4096, 8192, 16384: N = 128 6.1 6.6, 9.0 6.8, 14.9 7.0; N =
// 4096 6.6 7.5, 11.3 8.6, 21.0 12.9; at 64 rows N = 2048 7.9 10.3, 11.6 11.4, 24.4 16.2.
// Rows in no expert count as others do, and where one expert has them all the mean says
// little (gated, 2048 x 4096, one expert of 64 with all rows, and its matrix by itself):
// 512 rows 21.0 14.7, 4096 rows 71.0 46.3, 16384 rows 180 185.
ExpertTile expert_tile(int rows, int experts, int w_tiles, int k_tiles, int ctas) {
  const int active = std::max(1, std::min(rows, experts));
  const int each = (rows + experts - 1) / experts;
  const auto tiles = [&](int cols) {
    return static_cast<int64_t>(active) * ((each + cols - 1) / cols) * w_tiles;
  };
  // Whether cutting the few tiles there are saves more than the joining costs.
  const auto cuts = [&](int cols) {
    const int64_t pieces = std::min<int64_t>(ctas / tiles(cols), k_tiles / kMinPiece);
    return pieces > 1 && k_tiles - k_tiles / pieces >= (cols > 32 ? 40 : 24);
  };
  const auto of = [&](auto s, ExpertTile::Kind kind) {
    using S = decltype(s);
    return ExpertTile{kind, !S::kPair && cuts(S::kCols), S::kTiles, S::kXRows, S::kSmall};
  };
  const auto mean = [&](int64_t r) { return rows > r * experts; };
  if (!mean(16) || (2 * tiles(Narrow::kCols) <= ctas && k_tiles <= 32))
    return of(Narrow{}, ExpertTile::kNarrow);
  // (An odd tile of W leaves half a pair without one.)
  if (mean(64) &&
      tiles(Middle::kCols) * w_tiles > 2 * ctas * static_cast<int64_t>(w_tiles + w_tiles % 2))
    return of(Wide{}, ExpertTile::kWide);
  return of(Middle{}, ExpertTile::kMiddle);
}

cudaError_t launch_expert_product(const ExpertMaps& maps, const ExpertParams& p,
                                  const ExpertTile& tile, int ctas, cudaStream_t stream) {
  const auto as = [&](auto s, auto cuts) {
    using S = decltype(s);
    return p.gated ? launch_as<S, true, decltype(cuts)::value>(maps, p, ctas, stream)
                   : launch_as<S, false, decltype(cuts)::value>(maps, p, ctas, stream);
  };
  if (tile.kind == ExpertTile::kWide) return as(Wide{}, std::false_type{});
  if (tile.kind == ExpertTile::kMiddle)
    return tile.cuts ? as(Middle{}, std::true_type{}) : as(Middle{}, std::false_type{});
  return tile.cuts ? as(Narrow{}, std::true_type{}) : as(Narrow{}, std::false_type{});
}

cudaError_t launch_lay_scales(const uint8_t* scale, uint8_t* laid, int experts, int n, bool gated,
                              int w_tiles, int k_tiles, cudaStream_t stream) {
  lay_scales_kernel<<<dim3(k_tiles, w_tiles, experts), 128, 0, stream>>>(scale, laid, n, gated,
                                                                         w_tiles, k_tiles);
  return cudaGetLastError();
}

}  // namespace mxfp8
