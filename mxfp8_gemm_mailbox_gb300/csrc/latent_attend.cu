// Attention of a few query rows over a paged cache of latents, in the absorbed
// form: token p of a request is one vector c_p of `latent` numbers with a
// rotary key of 64 behind it, shared by every head, and is key and value at
// once,
//
//   z_p = scale (q . c_p),  e_p = exp(z_p - max z),
//   out = sum_p e_p c_p[0 : latent] / sum_p e_p        over the visible p.
//
// Request b has T = row_begin[b+1] - row_begin[b] query rows, its drafts, whose
// latents are the last T of its lengths[b] tokens.  Every row sees the tokens
// before them; among the drafts, row t sees draft j iff bit j of tree[t] is
// set (without a tree: iff j <= t).  A row that sees nothing gives zeros.
// Tokens past the length, and drafts that a row does not see, may hold
// anything, NaN included; a non-finite number in a draft's latent makes the
// rows that see it NaN.
//
// Mapping.  The T x heads rows of a request are packed into tiles of 128, the
// MMA's M.  128 rows x 512 FP32 outputs would take all of an SM's tensor
// memory, so a cluster of two CTAs shares a tile: CTA r holds columns
// [r latent/2, (r+1) latent/2) of the latent (and half of the rotary key) of
// every token, as key and as value, so a token crosses from L2 once per
// cluster.  Per tile of 64 tokens a CTA
//   1. multiplies its columns: partial scores of all 64 tokens;
//   2. sends the peer its partials of the peer's 32 tokens (FP32, distributed
//      shared memory) and adds the peer's partials of its own 32;
//   3. exponentiates its 32 and sends the peer their weights (BF16), straight
//      into the peer's MMA operand;
//   4. multiplies the weights of all 64 into its own output columns.
// The two halves exchange their maxima in a row tile's first token tile, whose
// common maximum becomes the row's reference (the exponent subtracted from its
// scores).  Later each half moves the reference it knows by whole steps alone,
// and the two agree on the larger afterwards: weights formed under different
// ones differ by a power of two, so bringing them together rounds nothing.
//
// Work.  The row tiles' token tiles are dealt to the clusters in runs: whole
// pieces of one row tile each where that costs little more than an even deal,
// else equal runs of the whole list.  A row tile cut between clusters leaves
// FP32 partial outputs with their references and sums, which a second kernel
// joins in a fixed order.
//
// Warps of a CTA:
//   0, 3   producers: TMA boxes into a ring, a lane a box: a row tile's queries
//          in two places of it, then its token tiles; a warp every other place
//          (a place costs its warp 0.5 to 1.2 us of look-ups and issue);
//   1      MMA issuer;
//   2      mender of the tiles that reach the drafts or the length: zeroes the
//          tokens past the length and drafts that are not finite;
//   4-11   softmax, two groups of four that take the token tiles in turn, so
//          one group's exchanges run under the other's: thread = row.
//
// Precision: scores, references, sums, outputs and partials FP32; the weights
// are rounded to BF16, the MMA's operand type (2^-8 relative at most), and the
// normaliser sums the rounded ones, so the weights that are applied sum to 1.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstddef>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kRope = 64;
constexpr int kTokens = 64;     // tokens in a tile
constexpr int kTileRows = 128;  // rows in a tile
constexpr int kMinBox = 8;      // tokens of a TMA box at least: pages are multiples of 8
constexpr int kAttendThreads = 384;
constexpr int kSoftmaxWarp = 4;
constexpr int kMaxRequests = MXFP8_MAX_REQUESTS;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
// A new maximum moves the reference of a row's exponentials only when it
// passes it by this many powers of two: the weights then stay below 2^9, far
// inside FP32 and BF16, and the outputs in tensor memory are seldom rescaled.
constexpr float kLazy = 8.0f;
// Pieces of one row tile a cluster may be this many token tiles longer than an
// even deal's runs: about what a second row tile in a run costs.
constexpr int kPieceSlack = 5;
constexpr int kMinRun = 2;
constexpr uint32_t kAtomBytes = kTokens * 128;  // 64 tokens x 64 columns
constexpr uint32_t kRopeBytes = kTokens * 64;   // 64 tokens x 32 rotary columns
constexpr uint32_t kQAtomBytes = kTileRows * 128;
constexpr uint32_t kQRopeBytes = kTileRows * 64;
// A group's partial scores from the peer (128 rows x 32 tokens x 4 bytes), then,
// read out, its weights (128 rows x 64 tokens x 2 bytes, swizzled): either way
// a quarter of 32 rows keeps to its own 4096 bytes.
constexpr uint32_t kExchangeBytes = kTileRows * 128;

template <int kLatent>
struct Shape {
  static constexpr int kHalf = kLatent / 2;  // columns of a CTA
  static constexpr int kAtoms = kHalf / 64;
  static constexpr uint32_t kStageBytes = kAtoms * kAtomBytes + kRopeBytes;
  static constexpr int kStages = kLatent == 512 ? 5 : 8;
  // Tensor-memory columns: outputs, queries (two BF16 a column), two score
  // tiles.
  static constexpr uint32_t kQ = kHalf;
  static constexpr uint32_t kS = kHalf + kHalf / 2;
  // Shared memory: the ring; the two groups' exchanges; the rotary part of the
  // queries.
  static constexpr uint32_t kX = kStages * kStageBytes;
  static constexpr uint32_t kQRope = kX + 2 * kExchangeBytes;
  static constexpr uint32_t kMisc = kQRope + kQRopeBytes;
  static_assert(kS + 2 * kTokens <= 512, "tensor memory");
  static_assert(kAtoms / 2 * kQAtomBytes + kQRopeBytes / 2 == kStageBytes,
                "half of the queries fill a place of the ring");
};

constexpr int kMaxStages = 8;
struct Misc {
  // Barriers, in four runs by their arrivals a phase.  Every one but `drained`
  // completes once a use, in order.
  uint64_t kv_full[kMaxStages], kv_ready[kMaxStages];    // 1 arrival
  uint64_t s_full[2], pv_done[2];                        // [tile parity]
  uint64_t recv[2][4], recv_credit[2][4];                // [group][lane quarter]
  uint64_t weights[2][4], weights_credit[2][4], decided[2][4];
  uint64_t tops[4];                                      // [lane quarter]
  uint64_t drained;
  uint64_t kv_empty[kMaxStages];                         // 2: outputs' commit, mender
  uint64_t s_free[2], p_full[2];                         // 4: the group's warps
  uint64_t q_ready;                                      // 8: all softmax warps
  uint64_t bad[kMaxStages];  // non-finite drafts of a stage's tile, one bit a token
  uint32_t tmem;
  int32_t abort;
  int32_t piece;  // token tiles of a piece, 0 for an even deal
  float peer_top[kTileRows];         // the peer's maxima in the first tile
  float reference[2][kTileRows];     // [tile parity][row], after that tile
  float2 peer[2][kTileRows];         // [group][row]: (reference, sum) of the peer's tokens
  uint32_t first[kMaxRequests + 1];  // runs (pieces, or token tiles) before each request
  int32_t length[kMaxRequests];
  uint16_t begin[kMaxRequests + 1];  // rows are at most MXFP8_MAX_LATENT_ROWS
};

// The device-side inputs of one request, cut to what the buffers hold.
struct Request {
  int begin, drafts, length;
  bool cut;
};
__device__ __forceinline__ Request load_request(const LatentParams& p, int b) {
  const int begin = p.row_begin[b], end = p.row_begin[b + 1], length = p.lengths[b];
  Request r;
  r.begin = min(max(begin, 0), p.rows);
  r.drafts = max(min(max(end, 0), p.rows) - r.begin, 0);
  r.length = min(max(length, 0), p.table_width * p.page_size);
  r.cut = begin < 0 || end > p.rows || end < begin || length != r.length;
  return r;
}
__device__ __forceinline__ int row_tiles(int drafts, int heads) {
  return (drafts * heads + kTileRows - 1) / kTileRows;
}
__device__ __forceinline__ int token_tiles(int length) {
  return (length + kTokens - 1) / kTokens;
}
__device__ __forceinline__ void raise(int32_t* flags, uint32_t bit) {
  if (flags != nullptr) atomicOr(reinterpret_cast<unsigned int*>(flags), bit);
}
__device__ __forceinline__ uint64_t low_ones(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(from - to) for references from <= to; equal infinities give 1.
__device__ __forceinline__ float shift_factor(float from, float to) {
  return from == to ? 1.0f : exp2_approx(from - to);
}
// Pairs of FP32 numbers in one instruction, each as the single one rounds.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t scale_bf16(uint32_t w, float f) {
  return pack_bf16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
}

__device__ __forceinline__ int drafts_of(const Misc& m, int b) {
  return max(m.begin[b + 1] - m.begin[b], 0);
}

// One row tile's run of token tiles inside a cluster's share.
struct Segment {
  int b, kv0, kv1, kv_tiles;
  int length, context, drafts, begin;
  int row0;   // first row of the tile within the request (drafts x heads rows)
  int valid;  // rows of the tile, at most 128
  int slot;   // of its partial outputs
};
struct Walk {
  uint32_t at, end, from;  // of the list of runs
  int b;
};
__device__ __forceinline__ bool next_segment(const Misc& m, const LatentParams& p, int cluster,
                                             Walk& w, Segment& s) {
  if (w.at >= w.end) return false;
  while (w.at >= m.first[w.b + 1]) ++w.b;
  s.b = w.b;
  s.length = m.length[w.b];
  s.begin = m.begin[w.b];
  s.drafts = drafts_of(m, w.b);
  s.context = max(s.length - s.drafts, 0);
  s.kv_tiles = token_tiles(s.length);
  const uint32_t local = w.at - m.first[w.b];
  int tile;
  if (m.piece > 0) {
    // At most as many pieces as clusters, so the products stay below 2^32.
    const uint32_t kv = s.kv_tiles, piece = m.piece;
    const uint32_t pieces = (kv + piece - 1) / piece;
    tile = local / pieces;
    const uint32_t k = local - tile * pieces;
    s.kv0 = kv * k / pieces;
    s.kv1 = kv * (k + 1) / pieces;
    s.slot = 2 * cluster;
    ++w.at;
  } else {
    const uint32_t kv = s.kv_tiles;
    tile = local / kv;
    s.kv0 = local - tile * kv;
    s.kv1 = min(s.kv_tiles, s.kv0 + static_cast<int>(w.end - w.at));
    // Only a share's first and last row tiles can be cut.
    s.slot = 2 * cluster + (w.at == w.from ? 0 : 1);
    w.at += s.kv1 - s.kv0;
  }
  s.row0 = tile * kTileRows;
  s.valid = min(kTileRows, s.drafts * p.heads - s.row0);
  return true;
}
// Whether a token tile reaches the drafts or the length.
__device__ __forceinline__ bool special(const Segment& s, int kv) {
  return (kv + 1) * kTokens > s.context;
}

// Bounded waits of a warp's lanes, which come out together.  One that runs out sets `abort`,
// after which every wait of the CTA returns at once and the kernel ends with
// its flag set.  (The softmax warps then run their loops out on whatever the
// buffers hold, so that none is missing at their barriers.)
struct Waiter {
  int32_t* abort;
  int32_t* flags;
  __device__ __forceinline__ bool operator()(const uint64_t& b, uint32_t parity) const {
    const uint32_t bar = ptx::smem_addr(&b);
    bool done = ptx::mbar_try_wait(bar, parity & 1u);
    if (!done) done = slow(bar, parity & 1u, false);
    __syncwarp();
    return done;
  }
  // With acquire over the cluster, for what a peer CTA signals.
  __device__ __forceinline__ bool cluster(const uint64_t& b, uint32_t parity) const {
    const uint32_t bar = ptx::smem_addr(&b);
    bool done = ptx::mbar_try_wait_cluster(bar, parity & 1u);
    if (!done) done = slow(bar, parity & 1u, true);
    __syncwarp();
    return done;
  }
  // Whether it is over already.
  __device__ __forceinline__ bool ready(const uint64_t& b, uint32_t parity) const {
    return __all_sync(~0u, ptx::mbar_test_wait(ptx::smem_addr(&b), parity & 1u));
  }
  // For a loop over ready(): whether it may go on after `spins` empty rounds
  // since `start` (set at the first).
  __device__ __noinline__ bool patient(int spins, uint64_t& start) const {
    const uint64_t now = ptx::globaltimer();
    if (spins == 0) start = now;
    if (*reinterpret_cast<volatile int32_t*>(abort) != 0) return false;
    if (now - start <= kWaitLimitNs) return true;
    *reinterpret_cast<volatile int32_t*>(abort) = 1;
    raise(flags, MXFP8_FLAG_GEMM_TIMEOUT);
    return false;
  }
  __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity, bool wide) const {
    uint64_t start = 0;
    for (int i = 0;; ++i) {
      if (wide ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity))
        return true;
      if (i % 16 == 0 && !patient(i, start)) return false;
    }
  }
};

struct AttendParams {
  LatentParams in;
  int32_t clusters;
  int32_t box;        // tokens of a TMA box: the largest of 64, 32, 16, 8 in a page
  float4* partial;    // [2 clusters][latent / 4][128 rows] x 4 columns
  float2* stats;      // [2 clusters][128 rows] (reference, sum)
  int32_t* piece;     // the deal: token tiles of a piece, 0 for equal runs
};
struct AttendMaps {
  CUtensorMap latent, rope;  // boxes of `box` tokens
  CUtensorMap q, q_rope;     // boxes of 128 and of 64 rows
};

// Token tiles of a cluster's run in an even deal.
__device__ __forceinline__ uint32_t run_length(uint32_t tiles, int clusters) {
  return max(static_cast<uint32_t>(kMinRun), (tiles + clusters - 1) / clusters);
}

// The deal, by one warp: fills Misc's lists.  (The host has checked that all
// token tiles number less than 2^31.)
__device__ __forceinline__ void deal(Misc& m, const AttendParams& ap, int lane) {
  const LatentParams& p = ap.in;
  uint32_t before = 0;
  int tiles_of_rows = 0;
  auto list = [&](int b, uint32_t runs) {  // sums of `runs` over the requests up to b
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(~0u, runs, o);
      if (lane >= o) runs += v;
    }
    if (b < p.requests) m.first[b + 1] = before + runs;
    before += __shfl_sync(~0u, runs, 31);
  };
  for (int base = 0; base < p.requests; base += 32) {
    const int b = base + lane;
    uint32_t tiles = 0;
    int rt = 0;
    if (b < p.requests) {
      const Request r = load_request(p, b);
      if (r.cut && blockIdx.x == 0) raise(p.flags, MXFP8_FLAG_BAD_INDEX);
      m.length[b] = r.length;
      m.begin[b] = static_cast<uint16_t>(r.begin);
      if (b == p.requests - 1) m.begin[b + 1] = static_cast<uint16_t>(r.begin + r.drafts);
      rt = r.length > 0 ? row_tiles(r.drafts, p.heads) : 0;
      tiles = static_cast<uint32_t>(rt) * token_tiles(r.length);
    }
    tiles_of_rows += __reduce_add_sync(~0u, rt);
    list(b, tiles);
  }
  // Pieces: the shortest length, from that of the even deal on, at which all
  // pieces fit the clusters, one a cluster; a lane a length.
  const int run = static_cast<int>(run_length(before, ap.clusters));
  int piece = 0;
  __syncwarp();
  if (tiles_of_rows <= ap.clusters) {
    int pieces = 0;
    if (lane <= kPieceSlack)
      for (int b = 0; b < p.requests; ++b)
        pieces += row_tiles(drafts_of(m, b), p.heads) *
                  ((token_tiles(m.length[b]) + run + lane - 1) / (run + lane));
    const uint32_t fits = __ballot_sync(~0u, lane <= kPieceSlack && pieces <= ap.clusters);
    if (fits != 0u) piece = run + __ffs(fits) - 1;
  }
  if (piece > 0) {
    before = 0;
    for (int base = 0; base < p.requests; base += 32) {
      const int b = base + lane;
      list(b, b < p.requests ? row_tiles(drafts_of(m, b), p.heads) *
                                   ((token_tiles(m.length[b]) + piece - 1) / piece)
                             : 0);
    }
  }
  if (lane == 0) {
    m.first[0] = 0;
    m.piece = piece;
    if (blockIdx.x == 0) *ap.piece = piece;
  }
}

template <int kLatent>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendMaps maps,
                  const __grid_constant__ AttendParams ap) {
  using L = Shape<kLatent>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = ptx::smem_addr(smem);
  Misc& m = *reinterpret_cast<Misc*>(smem + L::kMisc);
  const LatentParams& p = ap.in;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = ptx::cluster_ctarank();
  const int cluster = blockIdx.x / 2;
  auto bar = [&](const uint64_t& b) { return ptx::smem_addr(&b); };
  if (sbase % 1024u != 0) {  // the swizzles count from 1024-byte boundaries
    raise(p.flags, MXFP8_FLAG_GEMM_TIMEOUT);
    return;
  }

  if (warp == 0) {
    constexpr int kTwo = offsetof(Misc, kv_empty) / 8, kFour = offsetof(Misc, s_free) / 8;
    constexpr int kEight = offsetof(Misc, q_ready) / 8;
    for (int i = lane; i <= kEight; i += 32)
      ptx::mbar_init(bar(m.kv_full[0]) + 8u * i, i < kTwo ? 1 : i < kFour ? 2 : i < kEight ? 4 : 8);
    if (lane == 0) m.abort = 0;
    ptx::fence_mbarrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&m.tmem), 512);
    ptx::tmem_relinquish();
  }
  if (warp == 2 && lane < 4)
    ptx::prefetch_tensormap(reinterpret_cast<const CUtensorMap*>(&maps) + lane);
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = m.tmem;
  ptx::grid_dependency_wait();
  // Past the wait: the join may read this kernel's inputs at once.
  if (tid == 0) ptx::launch_dependents();
  if (warp == 0) deal(m, ap, lane);
  __syncthreads();

  const uint32_t all = m.first[p.requests];
  const uint32_t run = m.piece > 0 ? 1 : run_length(all, ap.clusters);
  const uint32_t from = min(all, cluster * run);
  Walk walk{from, min(all, from + run), from, 0};
  Segment seg{};
  const Waiter wait{&m.abort, p.flags};

  if (warp == 0 || warp == 3) {
    // -------------------------------------------------------------- producer
    // A lane a box (one thread's copies are served one after another).  The
    // page of a lane's box is read one of this warp's tiles ahead.
    const int which = warp == 3;
    constexpr int kItems = (kTokens / kMinBox * (L::kAtoms + 1) + 31) / 32;  // of a lane
    const uint64_t keep = ptx::policy_evict_last();
    // The page of copy i of tile kv (box i / (atoms + 1)): in the pool, or past
    // it (then the copy fills zeros) for a box past the length.
    const int items = kTokens / ap.box * (L::kAtoms + 1);
    auto read_page = [&](int kv, int i) {
      const int token = kv * kTokens + i / (L::kAtoms + 1) * ap.box;
      if (i >= items || token >= seg.length) return p.pages;
      return p.table[static_cast<size_t>(seg.b) * p.table_width + token / p.page_size];
    };
    int r = 0;  // places of the ring, of both warps
    bool ok = true;
    auto place = [&](uint32_t& full) {  // place r, once it is free
      if (r >= kStages) ok = __all_sync(~0u, wait(m.kv_empty[r % kStages], r / kStages - 1));
      full = bar(m.kv_full[r % kStages]);
      if (ok && lane == 0) ptx::mbar_arrive_expect_tx(full, L::kStageBytes);
      __syncwarp();
      return ok;
    };
    while (ok && next_segment(m, p, cluster, walk, seg)) {
      uint32_t full;
      // The queries: half of this CTA's columns and half of the rows' rotary
      // part a place.
      for (int half = 0; half < 2; ++half, ++r) {
        if ((r & 1) != which) continue;
        if (!place(full)) break;
        const uint32_t dst = sbase + r % kStages * L::kStageBytes;
        const int row = seg.begin * p.heads + seg.row0;
        if (lane < L::kAtoms / 2)
          ptx::tma_load_2d(dst + lane * kQAtomBytes, &maps.q,
                           static_cast<int>(rank) * L::kHalf +
                               (half * (L::kAtoms / 2) + lane) * 64,
                           row, full, ptx::policy_evict_first());
        else if (lane == L::kAtoms / 2)
          ptx::tma_load_2d(dst + L::kAtoms * kAtomBytes, &maps.q_rope,
                           static_cast<int>(rank) * 32, row + half * 64, full,
                           ptx::policy_evict_first());
        __syncwarp();
      }
      if (!ok) break;
      // This warp's first token tile.
      const int first = seg.kv0 + ((r & 1) != which);
      int page[kItems];
#pragma unroll
      for (int k = 0; k < kItems; ++k)
        page[k] = first < seg.kv1 ? read_page(first, lane + 32 * k) : p.pages;
      const int r0 = r - seg.kv0;
      for (int kv = first; kv < seg.kv1; kv += 2) {
        r = r0 + kv;
        int next[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k)
          next[k] = kv + 2 < seg.kv1 ? read_page(kv + 2, lane + 32 * k) : p.pages;
        if (!place(full)) break;
        const uint32_t dst = sbase + r % kStages * L::kStageBytes;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          const int i = lane + 32 * k;
          if (i >= items) continue;
          const int at = i / (L::kAtoms + 1) * ap.box, atom = i % (L::kAtoms + 1);
          if (page[k] < 0 || page[k] >= p.pages) {
            if (kv * kTokens + at < seg.length) raise(p.flags, MXFP8_FLAG_BAD_INDEX);
            page[k] = p.pages;
          }
          const int slot = (kv * kTokens + at) % p.page_size;
          if (atom < L::kAtoms)
            ptx::tma_load_3d(dst + atom * kAtomBytes + at * 128, &maps.latent,
                             static_cast<int>(rank) * L::kHalf + atom * 64, slot, page[k], full,
                             keep);
          else
            ptx::tma_load_3d(dst + L::kAtoms * kAtomBytes + at * 64, &maps.rope,
                             static_cast<int>(rank) * 32, slot, page[k], full, keep);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kItems; ++k) page[k] = next[k];
      }
      r = r0 + seg.kv1;
    }
    // Copies in flight land before the CTA leaves: each was waited for by the
    // mender, which passes every place, unless a wait ran out.
    for (int i = max(0, r - kStages); !ok && i < r; ++i)
      ptx::mbar_wait(bar(m.kv_full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u,
                     kWaitLimitNs / 16);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The warp stays converged and one elected lane issues: 32 clocks a
    // 128 x 64 x 16 product with the queries in tensor memory, the rate of the
    // tensor core; from a branch on the lane number it took 46.
    constexpr uint32_t kScores = ptx::idesc_bf16(kTokens, false);
    constexpr uint32_t kOutputs = ptx::idesc_bf16(L::kHalf, true);
    const uint32_t q_rope = sbase + L::kQRope;
    int g = 0;  // token tiles before the segment
    int r = 0;  // places of the ring before its first token tile
    uint32_t segments = 0;
    bool ok = true;
    auto tile_bar = [&](int i) -> const uint64_t& {
      const int stage = (r + i) % kStages;
      return special(seg, seg.kv0 + i) ? m.kv_ready[stage] : m.kv_full[stage];
    };
    auto scores = [&](int i) {
      const int j = g + i, stage = (r + i) % kStages;
      ptx::tc_fence_after();
      const uint32_t kvb = sbase + stage * L::kStageBytes;
      const uint32_t d = tmem + L::kS + (j & 1) * kTokens;
      const uint32_t done = bar(m.s_full[j & 1]);
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < L::kHalf / 16; ++k)
          ptx::mma_f16_ts(d, tmem + L::kQ + k * 8,
                          ptx::desc_kmajor_sw128(kvb + (k / 4) * kAtomBytes + (k % 4) * 32),
                          kScores, k > 0);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          ptx::mma_f16_ss(d, ptx::desc_kmajor_sw64(q_rope + k * 32),
                          ptx::desc_kmajor_sw64(kvb + L::kAtoms * kAtomBytes + k * 32), kScores,
                          1u);
        ptx::mma_commit(done);
      }
      __syncwarp();
    };
    auto outputs = [&](int i) {
      const int j = g + i, stage = (r + i) % kStages;
      ptx::tc_fence_after();
      const uint32_t kvb = sbase + stage * L::kStageBytes;
      const uint32_t weights = sbase + L::kX + (j & 1) * kExchangeBytes;
      const uint32_t add = i > 0;
      const uint32_t empty = bar(m.kv_empty[stage]), done = bar(m.pv_done[j & 1]);
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < kTokens / 16; ++k)
          ptx::mma_f16_ss(tmem, ptx::desc_kmajor_sw128(weights + k * 32),
                          ptx::desc_mnmajor_sw128(kvb + k * 2048, kAtomBytes), kOutputs,
                          k > 0 ? 1u : add);
        ptx::mma_commit(empty);
        ptx::mma_commit(done);
      }
      __syncwarp();
    };
    while (ok && next_segment(m, p, cluster, walk, seg)) {
      ok = __all_sync(~0u, wait(m.q_ready, segments++));
      if (lane == 0) {  // every softmax warp has read the queries
        ptx::mbar_arrive(bar(m.kv_empty[r % kStages]));
        ptx::mbar_arrive(bar(m.kv_empty[(r + 1) % kStages]));
      }
      r += 2;
      const int tiles = seg.kv1 - seg.kv0;
      // Whichever is ready: the scores of tile s (its tokens there, and the
      // scores of tile s - 2 read out of their buffer) or the outputs of tile o
      // (its weights there).  Neither waits behind the other, so a late tile
      // does not keep an earlier one's place in the ring.
      int s = 0, o = 0, spins = 0;
      uint64_t start = 0;
      while (ok && o < tiles) {
        if (s < tiles && s <= o + 2 && wait.ready(tile_bar(s), (r + s) / kStages) &&
            (s < 2 || wait.ready(m.s_free[(g + s) & 1], (g + s - 2) >> 1))) {
          scores(s++);
          spins = 0;
        } else if (o < s && wait.ready(m.p_full[(g + o) & 1], (g + o) >> 1)) {
          outputs(o++);
          spins = 0;
        } else if (spins++ % 64 == 0) {
          ok = __all_sync(~0u, wait.patient(spins - 1, start));
        }
      }
      g += tiles;
      r += tiles;
    }
    // Nothing runs on when tensor memory is freed.
    if (ptx::elect_one()) ptx::mma_commit(bar(m.drained));
    __syncwarp();
    ptx::mbar_wait(bar(m.drained), 0, kWaitLimitNs);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- mender
    int r = 0;
    bool ok = true;
    while (ok && next_segment(m, p, cluster, walk, seg)) {
      for (int kv = seg.kv0 - 2; ok && kv < seg.kv1; ++kv, ++r) {  // two of queries first
        const int stage = r % kStages;
        ok = __all_sync(~0u, wait(m.kv_full[stage], r / kStages));
        if (!ok) break;
        if (kv >= seg.kv0 && special(seg, kv)) {
          uint8_t* kvp = smem + stage * L::kStageBytes;
          const int n0 = max(seg.context - kv * kTokens, 0);
          const int n1 = min(seg.length - kv * kTokens, kTokens);
          // A token's 128-byte rows hold their 16-byte chunks in swizzled order,
          // which neither a search nor a fill minds.
          uint64_t bad = 0;
          for (int n = n0; n < n1; ++n) {
            bool finite = true;
            if (lane < L::kAtoms * 8) {
              const uint4 v = *reinterpret_cast<const uint4*>(kvp + (lane / 8) * kAtomBytes +
                                                              n * 128 + (lane % 8) * 16);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                finite = finite && (w[q] & 0x7F80u) != 0x7F80u &&
                         (w[q] & 0x7F800000u) != 0x7F800000u;
            }
            if (!__all_sync(~0u, finite)) bad |= 1ull << n;
          }
          // Boxes past the length came as zeros; the rest of the last one is
          // filled here.
          const uint64_t fill =
              bad | (low_ones((n1 + ap.box - 1) / ap.box * ap.box) & ~low_ones(n1));
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (int n = lane / 8; n < kTokens; n += 4) {  // 8 lanes a token's row of 128 bytes
            if (!(fill >> n & 1)) continue;
#pragma unroll
            for (int atom = 0; atom < L::kAtoms; ++atom)
              *reinterpret_cast<uint4*>(kvp + atom * kAtomBytes + n * 128 + lane % 8 * 16) = zero;
            if (lane % 8 < 4)
              *reinterpret_cast<uint4*>(kvp + L::kAtoms * kAtomBytes + n * 64 + lane % 8 * 16) =
                  zero;
          }
          if (lane == 0) m.bad[stage] = bad;
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(m.kv_ready[stage]));
          ptx::mbar_arrive(bar(m.kv_empty[stage]));
        }
      }
    }
  } else if (warp >= kSoftmaxWarp) {
    // --------------------------------------------------------------- softmax
    const int group = (warp - kSoftmaxWarp) / 4;  // takes the tiles of this parity
    const int quarter = warp & 3;  // the 32 tensor-memory lanes this warp reaches
    const int row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t score = lanes + L::kS + group * kTokens;
    const uint32_t peer = rank ^ 1u;
    const uint32_t recv_offset =
        L::kX + group * kExchangeBytes + quarter * 4096u + lane * 16u;
    const float4* recv = reinterpret_cast<const float4*>(smem + recv_offset);
    // A row of weights is one 128-byte swizzled row: this CTA's 32 tokens are
    // chunks 4 rank .. 4 rank + 3, in its own operand and in the peer's.
    const uint32_t p_row = L::kX + group * kExchangeBytes + row * 128u;
    auto chunk_at = [&](uint32_t half, int c) { return ((half * 4u + c) ^ (row & 7u)) * 16u; };
    const uint64_t& recv_bar = m.recv[group][quarter];
    const uint64_t& weights_bar = m.weights[group][quarter];
    // The peer's copy of a shared-memory address is this much further.
    const uint32_t over = ptx::map_to_rank(sbase, peer) - sbase;
    auto there = [&](const auto& x) { return ptx::smem_addr(&x) + over; };
    uint32_t exchanges = 0;  // tiles this warp exchanged
    uint32_t decisions = 0;  // tiles of this quarter's rows, of both groups
    uint32_t firsts = 0;     // row tiles of this quarter
    int g = 0;               // token tiles before the segment
    int r = 0;               // places of the ring before its first token tile
    // The peer may send this group its scores; after that, a permit follows
    // every tile whose outputs are added (its weights lay where scores land).
    if (lane == 0) ptx::mbar_arrive_remote_relaxed(there(m.recv_credit[group][quarter]));
    for (uint32_t segments = 0; next_segment(m, p, cluster, walk, seg); ++segments) {
      const size_t q_row = static_cast<size_t>(seg.begin) * p.heads + seg.row0 + row;
      const bool mine = row < seg.valid;
      const bool active = quarter * 32 < seg.valid;  // of the warp
      const int tiles = seg.kv1 - seg.kv0;
      const int i0 = (g & 1) != group;  // this group's first tile
      // Queries, from the ring: half of this CTA's columns a group into tensor
      // memory, and half of a row's rotary part (already swizzled).
      wait(m.kv_full[r % kStages], r / kStages);
      wait(m.kv_full[(r + 1) % kStages], (r + 1) / kStages);
      if (active) {
        const uint8_t* src = smem + (r + group) % kStages * L::kStageBytes + row * 128;
#pragma unroll
        for (int half = 0; half < L::kAtoms / 2; ++half) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + half * kQAtomBytes +
                                                            ((i ^ (row & 7)) * 16));
            v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
          }
          ptx::tmem_st_32x32b_x32(lanes + L::kQ + (group * (L::kAtoms / 2) + half) * 32, v);
        }
        const uint8_t* rope = smem + (r + row / 64) % kStages * L::kStageBytes +
                              L::kAtoms * kAtomBytes + row % 64 * 64;
#pragma unroll
        for (int i = 2 * group; i < 2 * group + 2; ++i)
          *reinterpret_cast<uint4*>(smem + L::kQRope + row * 64 + i * 16) =
              *reinterpret_cast<const uint4*>(rope + i * 16);
        ptx::tmem_wait_st();
        ptx::fence_proxy_async_smem();
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(m.q_ready));
      r += 2;
      if (!active) {
        for (int i = i0; i < tiles; i += 2) {
          wait(m.s_full[group], (g + i) >> 1);
          if (lane == 0) {
            ptx::mbar_arrive(bar(m.s_free[group]));
            ptx::mbar_arrive(bar(m.p_full[group]));
          }
          // (The scores two tiles on may come before this tile's weights: no
          // second arrival at one phase.)
          wait(m.p_full[group], (g + i) >> 1);
        }
        // Not on to the next segment before every warp has come to this one.
        wait(m.q_ready, segments);
        g += tiles;
        r += tiles;
        continue;
      }
      // What this row sees of the drafts.
      const int t = (seg.row0 + row) / p.heads;
      const uint64_t tree =
          p.tree != nullptr && mine ? static_cast<uint64_t>(p.tree[seg.begin + t]) : 0;
      // After this group's last tile: the row's common reference, and this
      // CTA's tokens' sum under `base`.
      float known = -INFINITY, base = -INFINITY, total = 0.0f;

      for (int i = i0; i < tiles; i += 2, ++exchanges) {
        const int kv = seg.kv0 + i;
        const uint32_t decision = decisions + i;
        if (i > i0) {
          wait(m.pv_done[group], (g + i - 2) >> 1);
          if (lane == 0) ptx::mbar_arrive_remote_relaxed(there(m.recv_credit[group][quarter]));
        }
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(bar(recv_bar), 32u * 32u * 4u);
          ptx::mbar_arrive_expect_tx(bar(weights_bar), 32u * (64u + 8u));
          if (i == 0) ptx::mbar_arrive_expect_tx(bar(m.tops[quarter]), 32u * 4u);
        }
        wait(m.s_full[group], (g + i) >> 1);
        ptx::tc_fence_after();
        uint32_t other[32], own[32];
        ptx::tmem_ld_32x32b_x32(score + peer * 32, other);
        ptx::tmem_ld_32x32b_x32(score + rank * 32, own);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(m.s_free[group]));
        if (special(seg, kv)) {
          const int stage = (r + i) % kStages;
          wait(m.kv_ready[stage], (r + i) / kStages);
          const uint64_t bad = m.bad[stage];
          if (bad != 0) {
            const uint32_t bad_other = static_cast<uint32_t>(bad >> (32 * peer));
            const uint32_t bad_own = static_cast<uint32_t>(bad >> (32 * rank));
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if (bad_other >> c & 1u) other[c] = 0x7FC00000u;
              if (bad_own >> c & 1u) own[c] = 0x7FC00000u;
            }
          }
        }
        // Scores: the peer's tokens out, its partials of this CTA's in.
        wait.cluster(m.recv_credit[group][quarter], exchanges);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          ptx::st_async_remote_v4(sbase + recv_offset + over + c * 512,
                                  make_uint4(other[4 * c], other[4 * c + 1], other[4 * c + 2],
                                             other[4 * c + 3]),
                                  there(recv_bar));
        wait.cluster(recv_bar, exchanges);
        float z[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 x = recv[c * 32];
          const float2 lo = add2(make_float2(__uint_as_float(own[4 * c]),
                                             __uint_as_float(own[4 * c + 1])),
                                 make_float2(x.x, x.y));
          const float2 hi = add2(make_float2(__uint_as_float(own[4 * c + 2]),
                                             __uint_as_float(own[4 * c + 3])),
                                 make_float2(x.z, x.w));
          z[4 * c] = lo.x, z[4 * c + 1] = lo.y, z[4 * c + 2] = hi.x, z[4 * c + 3] = hi.y;
        }
        if (special(seg, kv)) {
          const int at = kv * kTokens;
          uint64_t sees;
          if (p.tree != nullptr) {
            const int shift = at - seg.context;
            sees = shift >= 64 ? 0 : shift >= 0 ? tree >> shift : shift > -64 ? tree << -shift : 0;
            sees |= low_ones(seg.context - at);
          } else {
            sees = low_ones(seg.context + t + 1 - at);
          }
          sees &= low_ones(seg.length - at);
          const uint32_t bits = static_cast<uint32_t>(sees >> (32 * rank));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(bits >> c & 1u)) z[c] = -INFINITY;
        }
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) tops[c] = max3(z[c], z[c + 4], z[c + 8]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tops[c] = max3(tops[c], z[c + 12], z[c + 16]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tops[c] = max3(tops[c], z[c + 20], z[c + 24]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tops[c] = fmaxf(tops[c], z[c + 28]);
        const float top =
            fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * p.scale_log2;
        // The received scores have returned their values (each went into the
        // maximum), so the peer's weights may come over them.  (A release here
        // would wait for this CTA's own stores to the peer: it cost 60 us of 320
        // on 8 x 64k tokens, 128 heads.)
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote_relaxed(there(m.weights_credit[group][quarter]));
        // Weights of this CTA's tokens: under the halves' common maximum in the
        // first tile, then under the last reference this group knows, or one
        // whole steps above it.
        float under;
        if (i == 0) {
          ptx::st_async_remote(there(m.peer_top[row]), __float_as_uint(top),
                               there(m.tops[quarter]));
          wait.cluster(m.tops[quarter], firsts);
          under = fmaxf(top, m.peer_top[row]);
          m.reference[decision & 1][row] = under;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(m.decided[decision & 1][quarter]));
        } else {
          if (i == 1) {
            wait(m.decided[(decision - 1) & 1][quarter], (decision - 1) >> 1);
            known = m.reference[(decision - 1) & 1][row];
          }
          under = !(top > known + kLazy)  ? known
                  : known == -INFINITY    ? ceilf(top)
                                          : known + ceilf(top - known);
        }
        total *= shift_factor(base, under);
        base = under;
        const float sub = under == -INFINITY ? 0.0f : under;
        uint32_t w[16];
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 by = make_float2(p.scale_log2, p.scale_log2), less = make_float2(-sub, -sub);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 x = fma2(make_float2(z[2 * c], z[2 * c + 1]), by, less);
          w[c] = pack_bf16(exp2_approx(x.x), exp2_approx(x.y));
          sum[c % 2] = add2(sum[c % 2], make_float2(__uint_as_float(w[c] << 16),
                                                    __uint_as_float(w[c] & 0xFFFF0000u)));
        }
        sum[0] = add2(sum[0], sum[1]);
        total += sum[0].x + sum[0].y;
        wait.cluster(m.weights_credit[group][quarter], exchanges);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          ptx::st_async_remote_v4(sbase + p_row + over + chunk_at(rank, c),
                                  make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]),
                                  there(weights_bar));
        ptx::st_async_remote_v2(there(m.peer[group][row]), __float_as_uint(base),
                                __float_as_uint(total), there(weights_bar));
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(smem + p_row + chunk_at(rank, c)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        // The row's reference after this tile: the largest of the one before
        // and the two halves'.
        float before = -INFINITY;
        if (i > 0) {
          wait(m.decided[(decision - 1) & 1][quarter], (decision - 1) >> 1);
          before = m.reference[(decision - 1) & 1][row];
        }
        wait.cluster(weights_bar, exchanges);
        const float theirs = m.peer[group][row].x;
        const float now = fmaxf(before, fmaxf(base, theirs));
        if (i > 0) m.reference[decision & 1][row] = now;
        // Seldom anything else: all three references are the same.
        if (__any_sync(~0u, now != base || now != theirs || (i > 0 && now != before))) {
          const float f_own = shift_factor(base, now), f_peer = shift_factor(theirs, now);
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c) {
            uint4* at = reinterpret_cast<uint4*>(smem + p_row + chunk_at(0, c));
            const float f = c / 4 == rank ? f_own : f_peer;
            const uint4 v = *at;
            *at = make_uint4(scale_bf16(v.x, f), scale_bf16(v.y, f), scale_bf16(v.z, f),
                             scale_bf16(v.w, f));
          }
          if (i > 0) {
            // The outputs so far, once the tile before has been added.
            const float f = shift_factor(before, now);
            wait(m.pv_done[group ^ 1], (g + i - 1) >> 1);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < L::kHalf; c += 32) {
              ptx::tmem_ld_32x32b_x32(lanes + c, own);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q) own[q] = __float_as_uint(__uint_as_float(own[q]) * f);
              ptx::tmem_st_32x32b_x32(lanes + c, own);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
          }
        }
        known = now;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (i > 0) ptx::mbar_arrive(bar(m.decided[decision & 1][quarter]));
          ptx::mbar_arrive(bar(m.p_full[group]));
        }
      }

      // The row tile's outputs: the last tile is decided, and added (in this
      // order: then the barrier of the additions is at most one phase ahead of
      // a look at its parity).
      const uint32_t last = decisions + tiles - 1;
      decisions += tiles;
      ++firsts;
      wait(m.decided[last & 1][quarter], last >> 1);
      wait(m.pv_done[(g + tiles - 1) & 1], (g + tiles - 1) >> 1);
      ptx::tc_fence_after();
      const float now = m.reference[last & 1][row];
      // The sums, of both groups and both halves, under it.  The groups' pass
      // through the place of the last tile's weights, which its outputs have read
      // and the peer has no permit for yet.
      float* sums = reinterpret_cast<float*>(smem + L::kX + ((g + tiles - 1) & 1) * kExchangeBytes +
                                             quarter * 4096) +
                    lane;
      total *= shift_factor(base, now);
      if (i0 < tiles) total += m.peer[group][row].y * shift_factor(m.peer[group][row].x, now);
      sums[group * 32] = i0 < tiles ? total : 0.0f;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
      total = sums[0] + sums[32];
      asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
      if (lane == 0 && i0 < tiles) ptx::mbar_arrive_remote_relaxed(there(m.recv_credit[group][quarter]));
      const bool whole = seg.kv0 == 0 && seg.kv1 == seg.kv_tiles;
      const int column0 = static_cast<int>(rank) * L::kHalf + group * (L::kHalf / 2);
      const float inverse = total == 0.0f ? 0.0f : 1.0f / total;
      if (!whole && rank == 0 && group == 0 && mine)
        ap.stats[seg.slot * kTileRows + row] = make_float2(now, total);
#pragma unroll 1
      for (int c = 0; c < L::kHalf / 2; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(lanes + group * (L::kHalf / 2) + c, v);
        ptx::tmem_wait_ld();
        if (!mine) continue;
        if (whole) {
          uint16_t* out = p.out + q_row * kLatent + column0 + c;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              w[q] = pack_bf16(__uint_as_float(v[16 * i + 2 * q]) * inverse,
                               __uint_as_float(v[16 * i + 2 * q + 1]) * inverse);
            ptx::st_v8(out + 16 * i, w);
          }
        } else {
          float4* part = ap.partial +
                         (static_cast<size_t>(seg.slot) * (kLatent / 4) + (column0 + c) / 4) *
                             kTileRows +
                         row;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part[i * kTileRows] =
                make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                            __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        }
      }
      g += tiles;
      r += tiles;
    }
  }

  // --------------------------------------------------------------- teardown
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // no CTA leaves while its peer may address it
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the partial outputs of the row tiles that several clusters shared, in
// the order of their tokens, and writes the zeros of rows without tokens.
// Block (tile, 8 columns): thread = row x 4 columns.
template <int kLatent>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttendParams ap) {
  ptx::launch_dependents();
  const LatentParams& p = ap.in;
  const int row = threadIdx.x % kTileRows;
  const int column = blockIdx.y * 8 + (threadIdx.x / kTileRows) * 4;
  const int lane = threadIdx.x % 32;
  Request mine{p.rows, 0, 0, false};  // the first 32 requests, a lane each
  if (lane < p.requests) mine = load_request(p, lane);
  ptx::grid_dependency_wait();
  const int piece = *ap.piece;
  // Where this block's row tile stands in the list of runs; a lane a request.
  uint32_t all = 0, begin = 0, end = 0;
  int tiles = 0, covered0 = p.rows, covered1 = p.rows, row0 = 0, valid = 0;
  for (int base = 0; base < p.requests; base += 32) {
    Request r = mine;
    if (base > 0) {
      r = Request{p.rows, 0, 0, false};
      if (base + lane < p.requests) r = load_request(p, base + lane);
    }
    const int rt = row_tiles(r.drafts, p.heads);
    // Runs that a row tile of the request makes up.
    int kt = token_tiles(r.length);
    if (piece > 0) kt = (kt + piece - 1) / piece;
    int tiles_to = rt;
    uint32_t runs_to = static_cast<uint32_t>(rt) * kt;
    for (int o = 1; o < 32; o *= 2) {
      const int t = __shfl_up_sync(~0u, tiles_to, o);
      const uint32_t n = __shfl_up_sync(~0u, runs_to, o);
      if (lane >= o) tiles_to += t, runs_to += n;
    }
    const int tile = static_cast<int>(blockIdx.x) - (tiles + tiles_to - rt);
    const uint32_t has = __ballot_sync(~0u, tile >= 0 && tile < rt);
    if (has != 0u) {
      const int from = __ffs(has) - 1;
      const uint32_t at = all + runs_to - static_cast<uint32_t>(rt) * kt +
                          static_cast<uint32_t>(tile) * kt;
      begin = __shfl_sync(~0u, at, from);
      end = begin + __shfl_sync(~0u, kt, from);
      row0 = __shfl_sync(~0u, r.begin * p.heads + tile * kTileRows, from);
      valid = __shfl_sync(~0u, r.drafts * p.heads - tile * kTileRows, from);
    }
    if (base == 0) covered0 = __shfl_sync(~0u, r.begin, 0);
    if (base + 32 >= p.requests)
      covered1 = __shfl_sync(~0u, r.begin + r.drafts, p.requests - 1 - base);
    tiles += __shfl_sync(~0u, tiles_to, 31);
    all += __shfl_sync(~0u, runs_to, 31);
  }
  const size_t out_row = static_cast<size_t>(row0) + row;
  auto write = [&](size_t at, float4 v) {
    *reinterpret_cast<uint2*>(p.out + at * kLatent + column) =
        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  };
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (blockIdx.x == gridDim.x - 1) {  // rows before the first request or past the last
    const size_t lo = static_cast<size_t>(covered0) * p.heads;
    const size_t hi = static_cast<size_t>(covered1) * p.heads;
    const size_t n = static_cast<size_t>(p.rows) * p.heads;
    for (size_t at = row; at < lo; at += kTileRows) write(at, zero);
    for (size_t at = hi + row; at < n; at += kTileRows) write(at, zero);
    return;
  }
  if (row >= valid) return;
  if (begin == end) {
    write(out_row, zero);
    return;
  }
  // The clusters that shared the row tile: its pieces', or those whose runs
  // meet it.
  const uint32_t run = piece > 0 ? 1 : run_length(all, ap.clusters);
  const uint32_t c0 = begin / run, c1 = (end - 1) / run;
  if (c0 == c1) return;  // one cluster wrote the whole
  auto slot_of = [&](uint32_t c) { return 2 * c + (c * run < begin ? 1 : 0); };
  // Eight clusters' loads at a time, under the largest reference so far.
  constexpr uint32_t kBatch = 8;
  float top = -INFINITY, total = 0.0f;
  float4 sum = zero;
  for (uint32_t c = c0; c <= c1; c += kBatch) {
    float2 st[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (uint32_t k = 0; k < kBatch; ++k) {
      st[k] = make_float2(-INFINITY, 0.0f);
      v[k] = zero;
      if (c + k > c1) continue;
      const uint32_t slot = slot_of(c + k);
      st[k] = ap.stats[slot * kTileRows + row];
      v[k] = ap.partial[(static_cast<size_t>(slot) * (kLatent / 4) + column / 4) * kTileRows + row];
    }
    float next = top;
#pragma unroll
    for (uint32_t k = 0; k < kBatch; ++k) next = fmaxf(next, st[k].x);
    const float keep = shift_factor(top, next);
    top = next;
    total *= keep;
    sum = make_float4(sum.x * keep, sum.y * keep, sum.z * keep, sum.w * keep);
#pragma unroll
    for (uint32_t k = 0; k < kBatch; ++k) {
      const float f = shift_factor(st[k].x, top);
      total = fmaf(f, st[k].y, total);
      sum.x = fmaf(f, v[k].x, sum.x), sum.y = fmaf(f, v[k].y, sum.y);
      sum.z = fmaf(f, v[k].z, sum.z), sum.w = fmaf(f, v[k].w, sum.w);
    }
  }
  const float inverse = total == 0.0f ? 0.0f : 1.0f / total;
  write(out_row, make_float4(sum.x * inverse, sum.y * inverse, sum.z * inverse, sum.w * inverse));
}

constexpr int kMaxDevicesTracked = 64;
// Clusters whose partials the workspace holds.
constexpr int kMaxClusters = 80;

template <int kLatent>
constexpr uint32_t smem_bytes() {
  static_assert(MXFP8_MAX_LATENT_ROWS <= 65535, "row numbers fit 16 bits");
  static_assert(Shape<kLatent>::kMisc + sizeof(Misc) <= 232448, "shared memory of a CTA");
  return Shape<kLatent>::kMisc + sizeof(Misc);
}

// Clusters that run at once on the current device, asked once.
template <int kLatent>
cudaError_t resident_clusters(int* out) {
  static std::mutex mutex;
  static int known[kMaxDevicesTracked] = {};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= kMaxDevicesTracked) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mutex);
  if (known[device] == 0) {
    e = cudaFuncSetAttribute(attend_kernel<kLatent>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes<kLatent>());
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kMaxClusters);
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = smem_bytes<kLatent>();
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, attend_kernel<kLatent>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    known[device] = std::min(n, kMaxClusters);
  }
  *out = known[device];
  return cudaSuccess;
}

CUresult encode_cache(CUtensorMap* map, const LatentParams& p, int first, int columns, int box,
                      int box_columns, CUtensorMapSwizzle swizzle) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t page =
      p.pages > 1 ? p.page_stride : static_cast<int64_t>(p.page_size) * p.token_stride;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(p.page_size),
                        static_cast<cuuint64_t>(p.pages)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.token_stride) * 2, page * 2};
  cuuint32_t boxes[3] = {static_cast<cuuint32_t>(box_columns), static_cast<cuuint32_t>(box), 1};
  cuuint32_t elem[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.cache + first), dims,
            strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// q [rows x heads][latent + 64].
CUresult encode_queries(CUtensorMap* map, const LatentParams& p, int latent, int first,
                        int columns, int box_columns, int box_rows,
                        CUtensorMapSwizzle swizzle) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return CUDA_ERROR_NOT_FOUND;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns),
                        static_cast<cuuint64_t>(p.rows) * p.heads};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(latent + kRope) * 2};
  cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box_columns),
                         static_cast<cuuint32_t>(box_rows)};
  cuuint32_t elem[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p.q + first), dims,
            strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int kLatent>
cudaError_t launch_impl(const LatentParams& p, void* workspace, cudaStream_t stream) {
  AttendParams ap{};
  ap.in = p;
  cudaError_t e = resident_clusters<kLatent>(&ap.clusters);
  if (e != cudaSuccess) return e;
  ap.box = kTokens;
  while (p.page_size % ap.box) ap.box /= 2;
  ap.partial = static_cast<float4*>(workspace);
  ap.stats = reinterpret_cast<float2*>(ap.partial + static_cast<size_t>(2) * kMaxClusters *
                                                        (kLatent / 4) * kTileRows);
  ap.piece = reinterpret_cast<int32_t*>(ap.stats + static_cast<size_t>(2) * kMaxClusters *
                                                       kTileRows);
  AttendMaps maps;
  constexpr CUtensorMapSwizzle k128 = CU_TENSOR_MAP_SWIZZLE_128B, k64 = CU_TENSOR_MAP_SWIZZLE_64B;
  if (encode_cache(&maps.latent, p, 0, kLatent, ap.box, 64, k128) != CUDA_SUCCESS ||
      encode_cache(&maps.rope, p, kLatent, kRope, ap.box, 32, k64) != CUDA_SUCCESS ||
      encode_queries(&maps.q, p, kLatent, 0, kLatent, 64, kTileRows, k128) != CUDA_SUCCESS ||
      encode_queries(&maps.q_rope, p, kLatent, kLatent, kRope, 32, kTileRows / 2, k64) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;

  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * ap.clusters));
  cfg.blockDim = dim3(kAttendThreads);
  cfg.dynamicSmemBytes = smem_bytes<kLatent>();
  e = cudaLaunchKernelEx(&cfg, attend_kernel<kLatent>, maps, ap);
  if (e != cudaSuccess) return e;
  // Row tiles of all requests at most, and one block for the rows of none.
  const int tiles = static_cast<int>(static_cast<int64_t>(p.rows) * p.heads / kTileRows) +
                    std::min(p.requests, p.rows) + 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), kLatent / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<kLatent>, ap);
}

}  // namespace

size_t latent_workspace_bytes(int latent) {
  return static_cast<size_t>(2) * kMaxClusters * kTileRows *
             (static_cast<size_t>(latent) * sizeof(float) + sizeof(float2)) +
         256;
}

cudaError_t launch_latent_attend(const LatentParams& p, int latent, void* workspace,
                                 cudaStream_t stream) {
  return latent == 512 ? launch_impl<512>(p, workspace, stream)
                       : launch_impl<256>(p, workspace, stream);
}

}  // namespace mxfp8
