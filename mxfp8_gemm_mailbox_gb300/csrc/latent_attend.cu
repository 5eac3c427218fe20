// Attention of a few query rows over a paged cache of latents, in the absorbed
// form: token p of a request is one vector c_p of `latent` numbers with a
// rotary key of 64 behind it, shared by every head, and is key and value at
// once,
//
//   z_p = scale (q . c_p),  e_p = exp(z_p - max z),
//   out = sum_p e_p c_p[0 : latent] / sum_p e_p        over the visible p.
//
// Request b has T = row_begin[b+1] - row_begin[b] query rows, its drafts, whose
// latents are the last T of its lengths[b] tokens (of fewer than T, the first
// drafts have none).  Every row sees the tokens before them; among the drafts,
// row t sees draft j iff bit j of tree[t] is set (without a tree: iff j <= t).  A
// row that sees nothing gives zeros, one whose scores are all -infinity NaN.
// Tokens past the length, and drafts that a row does not see, may hold
// anything, NaN included; a non-finite number in a draft's latent makes the
// rows that see it NaN.
//
// Mapping.  The T x heads rows of a request are packed into tiles of 128, the
// M of a pair's product: a cluster of two CTAs shares the tile, 64 rows each,
// whose 64 x 512 FP32 outputs take half of an SM's tensor memory (a lane holds
// half of a row's columns).  Per tile of 64 tokens the pair
//   1. multiplies queries and keys: each CTA brings 32 of the tokens, whole;
//   2. exponentiates: each CTA its rows, a thread half of a row's tokens;
//   3. multiplies weights and values: each CTA brings its half of the latent
//      columns, of all tokens.
// Of the values a CTA lacks the peer's tokens; they are fetched (from L2, where
// the peer has just brought them) over the half of its own tokens that only
// the keys' product reads, as soon as that product is done.  The two products'
// operands must lie at the same addresses in both CTAs: with the first half of
// the columns (and of the tokens) in the first half of a place, they do.
//
// Work.  The row tiles' token tiles are dealt to the clusters in runs: whole
// pieces of one row tile each where that costs little more than an even deal,
// else equal runs of the whole list.  A row tile cut between clusters leaves
// FP32 partial outputs with their references and sums, which a second kernel
// joins in a fixed order.
//
// Warps of a CTA:
//   0, 3   producers: TMA boxes into a ring, a row tile's queries in two places
//          of it, then its token tiles; a warp every other place;
//   1, 14  issuers, in the first CTA, of the pair's products: scores, outputs;
//   2, 13  menders, of keys and of values: they pass every tile on to the
//          issuers, after a look at the ones that reach the drafts or the length;
//   4-11   softmax, two groups of four that take the token tiles in turn;
//   12     fetches the values of the peer's tokens, and what the shared memory
//          holds of the queries.
//
// Bounds, measured (latent 512, contexts spread so that none lies in L2):
//   8 x 64k tokens, 128 heads: 120 us = 5.1 TB/s, 1.22 PFLOP/s; 16 heads 116 us.
//     The stream of tokens: 111 us without the values' second fetch, 104
//     without products either.
//   8 drafts in a tree on 16k tokens, 128 heads: 39.6 us = 0.92 PFLOP/s.  29
//     token tiles of 0.8 us, 4.5 us before the first scores, 7 in which 20 MB of
//     partial outputs go to L2 and are joined.  The products fill 1250 of a
//     tile's 1450 clocks: 24 of the scores' at 18 and 12 at 25 (these read their
//     queries from shared memory, 128 bytes a clock), 8 of the outputs' at 64.
//   8 x 4k tokens, 128 heads: 26 us, 8 tiles and the same ends.
//   1 x 100 tokens, 16 heads: 8.5 us, a chain of latencies.
// Two CTAs that share a row tile by columns and exchange partial scores took
// 1.3 to 1.5 us a tile (174, 57 and 28.5 us for the first three).
//
// Precision: scores, references, sums, outputs and partials FP32; the weights
// are rounded to BF16, the MMA's operand type (2^-8 relative at most), and the
// normaliser sums the rounded ones, so the weights that are applied sum to 1.
// Normwise error against 64 bits 0.0017 to 0.0020, of which the rounding of the
// result is 0.0016; weights in two BF16 parts would take a second product with
// the values, 512 of a tile's 1450 clocks.
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
constexpr int kCtaTokens = 32;  // of them, those a CTA brings as keys
constexpr int kTileRows = 128;  // rows in a tile
constexpr int kCtaRows = 64;
constexpr int kMinBox = 8;      // tokens of a TMA box at least: pages are multiples of 8
constexpr int kAttendThreads = 480;
constexpr int kSoftmaxWarp = 4;
constexpr int kFetchWarp = 12;
constexpr int kValueMender = 13;
constexpr int kOutputWarp = 14;
constexpr int kMaxRequests = MXFP8_MAX_REQUESTS;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
// A new maximum moves the reference of a row's exponentials (a score before its
// scale) only when it passes it by this many powers of two: the weights then stay below 2^9, far
// inside FP32 and BF16, and the outputs in tensor memory are seldom rescaled.
constexpr float kLazy = 8.0f;
// Pieces of one row tile a cluster may be this many token tiles longer than an
// even deal's runs: about what a second row tile in a run costs (queries, a cold
// start and outputs, some 6 us; 8 x 64k tokens: 123 us with one piece of 114
// tiles a cluster, 129 with even runs of 108).
constexpr int kPieceSlack = 7;
// Token tiles of a run at least: four take about as long as the join of two
// halves (3 x 2.5k tokens, latent 256: 14.0 us, 15.7 with runs of 2; one request
// of 4k tokens, 128 heads: 16.2 us, 16.7 with 3, 17.6 with 6).
constexpr int kMinRun = 4;
constexpr int kMaxClusters = 80;  // whose partials the workspace holds
constexpr uint32_t kBlockBytes = kCtaTokens * 128;  // 32 tokens x 64 columns
constexpr uint32_t kQBlockBytes = kCtaRows * 128;   // 64 rows x 64 columns
constexpr uint32_t kWeightBytes = kCtaRows * kTokens * 2;

template <int kLatent>
struct Shape {
  static constexpr int kBlocks = kLatent / 64;
  static constexpr int kHalf = kBlocks / 2;  // blocks of a CTA's value columns
  // A place of the ring: a CTA's tokens, blocks of 64 columns, the rotary one
  // last.
  static constexpr uint32_t kPlaceBytes = (kBlocks + 1) * kBlockBytes;
  static constexpr int kStages = kLatent == 512 ? 5 : 9;
  // Blocks of the queries in tensor memory (in both halves of the lanes); the
  // rest, the rotary one last, in shared memory.
  static constexpr int kTmemBlocks = kLatent == 512 ? 6 : 4;
  static constexpr int kSmemBlocks = kBlocks + 1 - kTmemBlocks;
  // Tensor-memory columns: outputs, queries (two BF16 a column), two score
  // tiles.
  static constexpr int kColumns = kLatent / 2;  // of a lane's outputs
  static constexpr uint32_t kQ = kColumns;
  static constexpr uint32_t kS = kQ + kTmemBlocks * 32;
  // Shared memory: the ring; the two groups' weights; queries.
  static constexpr uint32_t kP = kStages * kPlaceBytes;
  static constexpr uint32_t kQSmem = kP + 2 * kWeightBytes;
  static constexpr uint32_t kMisc = kQSmem + kSmemBlocks * kQBlockBytes;
  static_assert(kS + 2 * kCtaTokens <= 512, "tensor memory");
  static_assert(kTmemBlocks / 2 * kQBlockBytes <= kPlaceBytes,
                "half of tensor memory's queries fit a place of the ring");
};

// One row tile's run of token tiles inside a cluster's share.
struct Segment {
  int b, kv0, kv1, kv_tiles;
  int length, drafts, begin;
  int context;  // tokens before the drafts; below 0 where the first drafts have no token
  int row0;   // first row of the tile within the request (drafts x heads rows)
  int valid;  // rows of the tile, at most 128
  int slot;   // of its partial outputs
};
struct Walk {
  uint32_t at, end, from;  // of the list of runs
  int b;                   // -1 before the share's first segment
};
// The deal.
struct Lists {
  uint32_t first[kMaxRequests + 1];  // runs (pieces, or token tiles) before each request
  int32_t length[kMaxRequests];
  uint16_t begin[kMaxRequests + 1];  // rows are at most MXFP8_MAX_LATENT_ROWS
  int32_t piece;                     // token tiles of a piece, 0 for an even deal
  uint32_t run;                      // runs of the list a cluster has
  Segment head;                      // this cluster's first segment
  Walk walk;                         // past it
};

template <int kStages>
struct Misc {
  // Barriers, in runs by their arrivals a phase.  Every one completes once a
  // use, in order.  The issuers wait on the first CTA's, which both CTAs arrive
  // on; a commit arrives on both CTAs'.
  uint64_t kv_full[kStages], kv_empty[kStages];  // 1; [place of the ring]
  uint64_t qk_done[kStages], v_full[kStages];    // 1; [token tile mod kStages]
  uint64_t s_full[2], pv_done[2];                // 1; [tile parity]
  uint64_t decided[2][4];                        // 1; [tile parity][lane quarter]
  uint64_t q_full, drained[2];                   // 1
  uint64_t k_ready[kStages], v_ready[kStages];   // 2: the CTAs' menders
  uint64_t s_free[2], p_full[2];                 // 8: a group's warps in both CTAs
  uint64_t q_ready;                              // 16: all softmax warps of both
  uint32_t tmem;
  int32_t abort;
  float tops[2][2][128];             // [a group's tile parity][group][lane]: maxima
  float reference[2][128];           // [tile parity][lane], after that tile
  float sums[4][kCtaRows];           // [group, token half][row]
  Lists lists;
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
// 2^((from - to) scale) for references from <= to; equal infinities give 1.
__device__ __forceinline__ float shift_factor(float from, float to, float scale) {
  return from == to ? 1.0f : exp2_approx((from - to) * scale);
}
// The sum of a row's weights so far where every score that it sees is -infinity:
// the formula's -infinity + infinity, if none comes that is not.  (A row that
// sees nothing has 0; a later reference shifts either away.)
constexpr float kAllInfinite = -1.0f;
__device__ __forceinline__ float inverse_of(float total) {
  return total == 0.0f ? 0.0f : total < 0.0f ? NAN : 1.0f / total;
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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
__device__ __forceinline__ bool finite_bf16(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    finite = finite && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
  return finite;
}

// Divisions, which stand in the way of a call's first copies (a 32-bit one by a
// variable is some 200 clocks).  By a number that the host knows, of n < 2^31:
struct Divisor {
  uint32_t magic;  // ceil(2^shift / d)
  int32_t shift;   // 31 + ceil(log2 d): the quotient's error n (magic d - 2^shift) / (d 2^shift)
                   // stays below 1 / d
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * magic >> shift);
  }
};
Divisor divisor_of(int d) {
  int log = 0;
  while ((int64_t{1} << log) < d) ++log;
  const uint64_t power = uint64_t{1} << (31 + log);
  return {static_cast<uint32_t>((power + d - 1) / d), 31 + log};
}
// By a variable: the approximate quotient (2 units in the last place) of n < 2^21
// is off by one at most.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d) {
  if (n >= 1u << 21) return n / d;
  uint32_t q = static_cast<uint32_t>(__fdividef(static_cast<float>(n), static_cast<float>(d)));
  const int32_t rest = static_cast<int32_t>(n - q * d);
  if (rest < 0)
    --q;
  else if (rest >= static_cast<int32_t>(d))
    ++q;
  return q;
}

__device__ __forceinline__ int drafts_of(const Lists& l, int b) {
  return max(l.begin[b + 1] - l.begin[b], 0);
}

// The segment at a place of a cluster's share, by a whole warp.
struct Next {
  Segment s;
  Walk w;
};
__device__ __forceinline__ Next segment_at(const Lists& l, int requests, int heads, int cluster,
                                           Walk w) {
  // The request of run `at`: a lane looks at one of 32.
  for (;; w.b += 32) {
    const int b = w.b + threadIdx.x % 32;
    const uint32_t past = __ballot_sync(~0u, b < requests && l.first[b + 1] <= w.at);
    if (past == ~0u) continue;
    w.b += __popc(past);
    break;
  }
  Segment s;
  s.b = w.b;
  s.length = l.length[w.b];
  s.begin = l.begin[w.b];
  s.drafts = drafts_of(l, w.b);
  s.context = s.length - s.drafts;
  s.kv_tiles = token_tiles(s.length);
  const uint32_t local = w.at - l.first[w.b];
  int tile;
  if (l.piece > 0) {
    // At most as many pieces as clusters, so the products stay below 2^32.
    const uint32_t kv = s.kv_tiles, piece = l.piece;
    const uint32_t pieces = quotient(kv + piece - 1, piece);
    tile = quotient(local, pieces);
    const uint32_t k = local - tile * pieces;
    s.kv0 = quotient(kv * k, pieces);
    s.kv1 = quotient(kv * (k + 1), pieces);
    s.slot = 2 * cluster;
    ++w.at;
  } else {
    const uint32_t kv = s.kv_tiles;
    tile = quotient(local, kv);
    s.kv0 = local - tile * kv;
    s.kv1 = min(s.kv_tiles, s.kv0 + static_cast<int>(w.end - w.at));
    // Only a share's first and last row tiles can be cut.
    s.slot = 2 * cluster + (w.at == w.from ? 0 : 1);
    w.at += s.kv1 - s.kv0;
  }
  s.row0 = tile * kTileRows;
  s.valid = min(kTileRows, s.drafts * heads - s.row0);
  return {s, w};
}
// The first segment is found once, with the deal: with a copy of that code a
// role, the warps waited for it to come from far, 0.7 to 1.4 us.
__device__ __noinline__ Next step(const Lists& l, int requests, int heads, int cluster, Walk w) {
  return segment_at(l, requests, heads, cluster, w);
}
__device__ __forceinline__ bool next_segment(const Lists& l, const LatentParams& p, int cluster,
                                             Walk& w, Segment& s) {
  if (w.b < 0) {
    s = l.head;
    w = l.walk;
    return s.kv1 > s.kv0;
  }
  if (w.at >= w.end) return false;
  const Next next = step(l, p.requests, p.heads, cluster, w);
  s = next.s;
  w = next.w;
  return true;
}
// Whether a token tile reaches the drafts or the length.
__device__ __forceinline__ bool special(const Segment& s, int kv) {
  return (kv + 1) * kTokens > s.context;
}

// Bounded waits of a warp's lanes, which come out together.  One that runs out
// sets `abort`, after which every wait of the CTA returns at once and the
// kernel ends with its flag set.  (The softmax warps then run their loops out on whatever the
// buffers hold, so that none is missing at their barriers.)
struct Waiter {
  int32_t* abort;
  int32_t* flags;
  __device__ __forceinline__ bool operator()(const uint64_t& b, uint32_t parity) const {
    const uint32_t bar = ptx::smem_addr(&b);
    bool done = ptx::mbar_try_wait(bar, parity & 1u);
    if (!done) done = slow(bar, parity & 1u);
    __syncwarp();
    return done;
  }
  __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity) const {
    const uint64_t start = ptx::globaltimer();
    for (int i = 0;; ++i) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      if (i % 16 != 0) continue;
      if (*reinterpret_cast<volatile int32_t*>(abort) != 0) return false;
      if (ptx::globaltimer() - start <= kWaitLimitNs) continue;
      *reinterpret_cast<volatile int32_t*>(abort) = 1;
      raise(flags, MXFP8_FLAG_GEMM_TIMEOUT);
      return false;
    }
  }
};

// A row tile that begins in a cluster's share and ends in another's: its slot
// there, the last cluster (whose slot is its first, as are those between), its
// first row of all (rows x heads) and how many; 0 rows: none.
struct Cut {
  int32_t slot, last, row0, rows;
};
struct AttendParams {
  LatentParams in;
  int32_t clusters;
  int32_t box;        // tokens of a TMA box: the largest of 32, 16, 8 in a page
  int32_t box_log2;
  Divisor by_page, by_clusters;  // page_size, clusters
  float4* partial;    // [2 clusters][latent / 4][128 rows] x 4 columns
  float2* stats;      // [2 clusters][128 rows] (reference, sum)
  Cut* cuts;          // [clusters]
};
struct AttendMaps {
  // Boxes of 64 columns by `box` tokens (64 rows), by as many blocks of columns
  // as a copy takes.
  CUtensorMap keys, values, q;
};

// Token tiles of a cluster's run in an even deal.
__device__ __forceinline__ uint32_t run_length(uint32_t tiles, const AttendParams& ap) {
  return max(kMinRun, ap.by_clusters(tiles + ap.clusters - 1));
}

// The deal, by one warp.  (The host has checked that all token tiles number
// at most 2^30.)
__device__ __forceinline__ void deal(Lists& l, const AttendParams& ap, int cluster, int lane) {
  const LatentParams& p = ap.in;
  uint32_t all = 0;  // token tiles
  int tiles = 0;     // row tiles
  for (int base = 0; base < p.requests; base += 32) {
    const int b = base + lane;
    int rt = 0, tt = 0;
    if (b < p.requests) {
      const Request r = load_request(p, b);
      if (r.cut && blockIdx.x == 0) raise(p.flags, MXFP8_FLAG_BAD_INDEX);
      l.length[b] = r.length;
      l.begin[b] = static_cast<uint16_t>(r.begin);
      if (b == p.requests - 1) l.begin[b + 1] = static_cast<uint16_t>(r.begin + r.drafts);
      rt = r.length > 0 ? row_tiles(r.drafts, p.heads) : 0;
      tt = token_tiles(r.length);
    }
    all += __reduce_add_sync(~0u, static_cast<uint32_t>(rt) * tt);
    tiles += __reduce_add_sync(~0u, rt);
  }
  __syncwarp();
  // Rows given to several requests could make up more tiles than the host
  // counted: such a list is not dealt at all.
  const bool sound = tiles <= p.rows * p.heads / kTileRows + p.requests;
  if (!sound && blockIdx.x == 0 && lane == 0) raise(p.flags, MXFP8_FLAG_BAD_INDEX);
  auto row_tiles_of = [&](int b) {
    return sound && l.length[b] > 0 ? row_tiles(drafts_of(l, b), p.heads) : 0;
  };
  // Pieces: the shortest length, from that of the even deal on, at which all
  // pieces fit the clusters, one a cluster; a lane a length and every fourth
  // request.
  static_assert(kPieceSlack < 8, "");
  const uint32_t run = run_length(all, ap), slack = lane % 8;
  uint32_t piece = 0;
  if (tiles <= ap.clusters) {
    uint32_t pieces = 0;
    for (int b = lane / 8; b < p.requests; b += 4)
      pieces += row_tiles_of(b) * quotient(token_tiles(l.length[b]) + run + slack - 1, run + slack);
    pieces += __shfl_xor_sync(~0u, pieces, 8);
    pieces += __shfl_xor_sync(~0u, pieces, 16);
    const uint32_t fits = __ballot_sync(
        ~0u, slack <= kPieceSlack && pieces <= static_cast<uint32_t>(ap.clusters));
    if (fits != 0u) piece = run + __ffs(fits) - 1;
  }
  uint32_t before = 0;
  for (int base = 0; base < p.requests; base += 32) {
    const int b = base + lane;
    uint32_t runs = 0;
    if (b < p.requests) {
      const uint32_t tt = token_tiles(l.length[b]);
      runs = row_tiles_of(b) * (piece > 0 ? quotient(tt + piece - 1, piece) : tt);
    }
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(~0u, runs, o);
      if (lane >= o) runs += v;
    }
    if (b < p.requests) l.first[b + 1] = before + runs;
    before += __shfl_sync(~0u, runs, 31);
  }
  if (lane == 0) {
    l.first[0] = 0;
    l.piece = static_cast<int>(piece);
    l.run = piece > 0 ? 1 : run;
  }
  __syncwarp();
  const uint32_t share = piece > 0 ? 1 : run;
  const uint32_t from = min(before, cluster * share), end = min(before, from + share);
  Next next{{}, {from, end, from, 0}};
  if (from < end) next = segment_at(l, p.requests, p.heads, cluster, next.w);
  if (lane == 0) {
    l.head = next.s;
    l.walk = next.w;
  }
}

// Zeros for the rows before the first request, past the last and of requests
// without tokens; a warp of every cluster, in turn.
__device__ __forceinline__ void zero_rows(const Lists& l, const LatentParams& p, int lane,
                                          int latent) {
  auto zero = [&](int from, int to) {
    const int row_bytes = p.heads * latent * 2;  // a multiple of 512
    for (int t = from + blockIdx.x / 2; t < to; t += gridDim.x / 2) {
      uint4* row = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.out) +
                                            static_cast<size_t>(t) * row_bytes);
      for (int i = lane; i < row_bytes / 16; i += 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  zero(0, p.requests > 0 ? l.begin[0] : 0);
  zero(p.requests > 0 ? l.begin[p.requests] : 0, p.rows);
  for (int base = 0; base < p.requests; base += 32) {
    const int b = base + lane;
    uint32_t empty =
        __ballot_sync(~0u, b < p.requests && l.length[b] == 0 && drafts_of(l, b) > 0);
    for (; empty != 0u; empty &= empty - 1u) {
      const int e = base + __ffs(empty) - 1;
      zero(l.begin[e], l.begin[e + 1]);
    }
  }
}

template <int kLatent>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendMaps maps,
                  const __grid_constant__ AttendParams ap) {
  using L = Shape<kLatent>;
  constexpr int kStages = L::kStages;
  using Local = Misc<kStages>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = ptx::smem_addr(smem);
  Local& m = *reinterpret_cast<Local*>(smem + L::kMisc);
  const LatentParams& p = ap.in;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = ptx::cluster_ctarank();
  const int cluster = blockIdx.x / 2;
  auto bar = [&](const uint64_t& b) { return ptx::smem_addr(&b); };
  auto first_cta = [&](const uint64_t& b) { return ptx::map_to_rank(ptx::smem_addr(&b), 0); };
  if (sbase % 1024u != 0) {  // the swizzles count from 1024-byte boundaries
    raise(p.flags, MXFP8_FLAG_GEMM_TIMEOUT);
    return;
  }

  if (warp == 0) {
    constexpr int kTwo = offsetof(Local, k_ready) / 8, kEight = offsetof(Local, s_free) / 8;
    constexpr int kLast = offsetof(Local, q_ready) / 8;
    for (int i = lane; i <= kLast; i += 32)
      ptx::mbar_init(bar(m.kv_full[0]) + 8u * i, i < kTwo ? 1 : i < kEight ? 2 : i < kLast ? 8 : 16);
    if (lane == 0) m.abort = 0;
    ptx::fence_mbarrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(&m.tmem), 512);
    ptx::tmem_relinquish_pair();
  }
  if (warp == 2 && lane < 3)
    ptx::prefetch_tensormap(reinterpret_cast<const CUtensorMap*>(&maps) + lane);
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = m.tmem;
  // The wait for the kernel before and for the deal.  Every role makes it at its
  // own start: the code that follows is then at hand when it is over.
  auto begin = [&] {
    ptx::grid_dependency_wait();
    asm volatile("bar.sync 0;" ::: "memory");
  };

  Walk walk{0, 0, 0, -1};
  Segment seg{};
  const Waiter wait{&m.abort, p.flags};
  // The page of the box with token `token`: in the pool, or past it (then the
  // copy fills zeros) for a box past the length.
  auto read_page = [&](int token) {
    if (token >= seg.length) return p.pages;
    return p.table[static_cast<size_t>(seg.b) * p.table_width + ap.by_page(token)];
  };

  auto slot_of = [&](int token) { return token - ap.by_page(token) * p.page_size; };

  if (warp == 0 || warp == 3) {
    // -------------------------------------------------------------- producer
    if (warp == 0) {
      ptx::grid_dependency_wait();
      deal(m.lists, ap, cluster, lane);
    }
    begin();
    // A tile's part in one copy where a page holds 32 tokens in a row, else a
    // lane a box of each block.  The page of a lane's box is read one of this
    // warp's tiles ahead.
    const int which = warp == 3;
    constexpr int kItems = (kCtaTokens / kMinBox * (L::kBlocks + 1) + 31) / 32;  // of a lane
    const bool whole = ap.box == kCtaTokens;
    const int items = whole ? 1 : (kCtaTokens >> ap.box_log2) * (L::kBlocks + 1);
    auto box_of = [&](int i) { return whole ? 0 : i / (L::kBlocks + 1) << ap.box_log2; };
    // The first token of copy i of this CTA's part of tile kv.
    auto token_of = [&](int kv, int i) {
      return kv * kTokens + static_cast<int>(rank) * kCtaTokens + box_of(i);
    };
    auto page_of = [&](int kv, int i) {
      return kv < seg.kv1 && i < items ? read_page(token_of(kv, i)) : p.pages;
    };
    int r = 0;  // places of the ring, of both warps
    bool ok = true;
    auto place = [&](uint32_t bytes, uint32_t& full) {  // place r, once it is free
      if (r >= kStages) ok = __all_sync(~0u, wait(m.kv_empty[r % kStages], r / kStages - 1));
      full = bar(m.kv_full[r % kStages]);
      if (ok && lane == 0) ptx::mbar_arrive_expect_tx(full, bytes);
      __syncwarp();
      return ok;
    };
    while (ok && next_segment(m.lists, p, cluster, walk, seg)) {
      // This warp's first token tile.
      const int first = seg.kv0 + ((r & 1) != which);  // (the queries take two places)
      int page[kItems];
#pragma unroll
      for (int k = 0; k < kItems; ++k) page[k] = page_of(first, lane + 32 * k);
      uint32_t full;
      // The queries that go to tensor memory, half of their blocks a place.
      for (int half = 0; half < 2; ++half, ++r) {
        if ((r & 1) != which) continue;
        if (!place(L::kTmemBlocks / 2 * kQBlockBytes, full)) break;
        if (lane < L::kTmemBlocks / 2)
          ptx::tma_load_2d(sbase + r % kStages * L::kPlaceBytes + lane * kQBlockBytes, &maps.q,
                           (half * (L::kTmemBlocks / 2) + lane) * 64,
                           seg.begin * p.heads + seg.row0 + static_cast<int>(rank) * kCtaRows,
                           full, ptx::policy_evict_first());
        __syncwarp();
      }
      if (!ok) break;
      const int r0 = r - seg.kv0;
      for (int kv = first; kv < seg.kv1; kv += 2) {
        r = r0 + kv;
        int next[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) next[k] = page_of(kv + 2, lane + 32 * k);
        if (!place(L::kPlaceBytes, full)) break;
        const uint32_t dst = sbase + r % kStages * L::kPlaceBytes;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          const int i = lane + 32 * k;
          if (i >= items) continue;
          const int block = whole ? 0 : i % (L::kBlocks + 1), at = box_of(i);
          const int token = token_of(kv, i);
          if (page[k] < 0 || page[k] >= p.pages) {
            if (token < seg.length) raise(p.flags, MXFP8_FLAG_BAD_INDEX);
            page[k] = p.pages;
          }
          ptx::tma_load_4d(dst + block * kBlockBytes + at * 128, &maps.keys, 0,
                           slot_of(token), block, page[k], full);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kItems; ++k) page[k] = next[k];
      }
      r = r0 + seg.kv1;
    }
    // The first CTA's last release of each place has landed.
    for (int i = max(0, r - kStages); ok && i < r; ++i)
      if ((i & 1) == which) ok = __all_sync(~0u, wait(m.kv_empty[i % kStages], i / kStages));
    // Copies in flight land before the CTA leaves: each was waited for by the
    // mender, which passes every place, unless a wait ran out.
    for (int i = max(0, r - kStages); !ok && i < r; ++i)
      ptx::mbar_wait(bar(m.kv_full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u,
                     kWaitLimitNs / 16);
  } else if (warp == kFetchWarp) {
    // ----------------------------------------------------------------- fetch
    begin();
    // This CTA's value columns of the peer's tokens, over the blocks of its own
    // tokens that only the keys' product reads.
    const bool whole = ap.box == kCtaTokens;
    const int items = whole ? 1 : (kCtaTokens >> ap.box_log2) * L::kHalf;  // at most 16
    const int block = whole ? 0 : lane % L::kHalf;
    const int at = whole ? 0 : lane / L::kHalf << ap.box_log2;
    const int column0 = static_cast<int>(rank) * L::kHalf, theirs = static_cast<int>(rank ^ 1u);
    auto token_of = [&](int kv) {
      return kv * kTokens + theirs * kCtaTokens + at;
    };
    auto page_of = [&](int kv) {
      return kv < seg.kv1 && lane < items ? read_page(token_of(kv)) : p.pages;
    };
    int r = 0, j = 0;  // places of the ring, token tiles
    uint32_t segments = 0;
    bool ok = true;
    for (; ok && next_segment(m.lists, p, cluster, walk, seg); ++segments) {
      // Every product with the last row tile's queries is done.
      const uint32_t full = bar(m.q_full);
      if (lane == 0) ptx::mbar_arrive_expect_tx(full, L::kSmemBlocks * kQBlockBytes);
      __syncwarp();
      if (lane < L::kSmemBlocks)
        ptx::tma_load_2d(sbase + L::kQSmem + lane * kQBlockBytes, &maps.q,
                         (L::kTmemBlocks + lane) * 64,
                         seg.begin * p.heads + seg.row0 + static_cast<int>(rank) * kCtaRows, full,
                         ptx::policy_evict_first());
      __syncwarp();
      r += 2;
      int page = page_of(seg.kv0);
      for (int kv = seg.kv0; kv < seg.kv1; ++kv, ++r, ++j) {
        const int next = page_of(kv + 1);
        ok = __all_sync(~0u, wait(m.qk_done[j % kStages], j / kStages));
        if (!ok) break;
        const uint32_t done = bar(m.v_full[j % kStages]);
        if (lane == 0) ptx::mbar_arrive_expect_tx(done, L::kHalf * kBlockBytes);
        __syncwarp();
        if (lane < items) {
          if (page < 0 || page >= p.pages) page = p.pages;
          ptx::tma_load_4d(sbase + r % kStages * L::kPlaceBytes +
                               (theirs * L::kHalf + block) * kBlockBytes + at * 128,
                           &maps.values, 0, slot_of(token_of(kv)), column0 + block, page,
                           done);
        }
        __syncwarp();
        page = next;
      }
    }
    if (!ok) {
      if (segments > 0) ptx::mbar_wait(bar(m.q_full), (segments - 1) & 1u, kWaitLimitNs / 16);
      for (int i = max(0, j - kStages); i < j; ++i)
        ptx::mbar_wait(bar(m.v_full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u,
                       kWaitLimitNs / 16);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- scores' issuer
    begin();
    // Both issuers stay converged and one elected lane issues (from a branch on
    // the lane number a product took half as long again).  A pair's 128 x 64 x
    // 16 product takes 18 clocks with the queries in tensor memory, 25 with
    // them in shared memory; 128 x 256 x 16 takes 64, the tensor cores' rate.
    // One warp for both products left the tensor cores idle while it looked
    // for the next that was ready: 0.2 us a look.
    constexpr uint32_t kScores = ptx::idesc_bf16(kTokens, false);
    int j = 0;  // token tiles
    int r = 0;  // places of the ring
    uint32_t segments = 0;
    bool ok = rank == 0;
    while (ok && next_segment(m.lists, p, cluster, walk, seg)) {
      ok = __all_sync(~0u, wait(m.q_ready, segments++));
      // Every softmax warp has read the queries.
      if (lane < 4)
        ptx::mbar_arrive_remote(
            ptx::map_to_rank(bar(m.kv_empty[(r + lane / 2) % kStages]), lane % 2));
      __syncwarp();
      r += 2;
      for (int kv = seg.kv0; ok && kv < seg.kv1; ++kv, ++r, ++j) {
        // The tile's tokens are there, and the scores of the one before the
        // last are read out of their buffer.
        ok = wait(m.k_ready[j % kStages], j / kStages);
        if (kv >= seg.kv0 + 2) ok = wait(m.s_free[j & 1], (j - 2) >> 1) && ok;
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t keys = sbase + r % kStages * L::kPlaceBytes;
        const uint32_t d = tmem + L::kS + (j & 1) * kCtaTokens;
        const uint32_t done = bar(m.s_full[j & 1]), fetch = bar(m.qk_done[j % kStages]);
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < L::kTmemBlocks * 4; ++k)
            ptx::mma_f16_ts_pair(
                d, tmem + L::kQ + k * 8,
                ptx::desc_kmajor_sw128(keys + (k / 4) * kBlockBytes + (k % 4) * 32), kScores, k > 0);
#pragma unroll
          for (int k = 0; k < L::kSmemBlocks * 4; ++k)
            ptx::mma_f16_ss_pair(
                d,
                ptx::desc_kmajor_sw128(sbase + L::kQSmem + (k / 4) * kQBlockBytes + (k % 4) * 32),
                ptx::desc_kmajor_sw128(keys + (L::kTmemBlocks + k / 4) * kBlockBytes +
                                       (k % 4) * 32),
                kScores, 1u);
          ptx::mma_commit_pair(fetch);
          ptx::mma_commit_pair(done);
        }
        __syncwarp();
      }
    }
    if (rank == 0) {
      // The softmax warps' last arrivals, which no product waits for.
      for (int i = max(0, j - 2); ok && i < j; ++i)
        ok = __all_sync(~0u, wait(m.s_free[i & 1], i >> 1));
      if (ptx::elect_one()) ptx::mma_commit_pair(bar(m.drained[0]));
    }
  } else if (warp == kOutputWarp) {
    // -------------------------------------------------------- outputs' issuer
    begin();
    if (rank == 1) {  // nothing to issue
      zero_rows(m.lists, p, lane, kLatent);
      // For the join.
      Cut cut{0, 0, 0, 0};
      Walk ahead = walk;
      for (;;) {
        if (!next_segment(m.lists, p, cluster, ahead, seg)) break;
        if (seg.kv0 != 0 || seg.kv1 == seg.kv_tiles) continue;
        // The clusters of its other runs follow this one.
        const int piece = m.lists.piece, left = seg.kv_tiles - seg.kv1;
        const int more = piece > 0 ? (seg.kv_tiles + piece - 1) / piece - 1
                                   : (left + m.lists.run - 1) / m.lists.run;
        cut = Cut{seg.slot, cluster + more, seg.begin * p.heads + seg.row0, seg.valid};
      }
      if (lane == 0) ap.cuts[cluster] = cut;
    }
    constexpr uint32_t kOutputs = ptx::idesc_bf16(256, true);
    int j = 0, r = 0;
    bool ok = rank == 0;
    while (ok && next_segment(m.lists, p, cluster, walk, seg)) {
      r += 2;
      for (int kv = seg.kv0; ok && kv < seg.kv1; ++kv, ++r, ++j) {
        ok = wait(m.v_ready[j % kStages], j / kStages);
        ok = wait(m.p_full[j & 1], j >> 1) && ok;
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const int stage = r % kStages;
        const uint32_t values = sbase + stage * L::kPlaceBytes;
        const uint32_t weights = sbase + L::kP + (j & 1) * kWeightBytes;
        const uint32_t add = kv > seg.kv0;
        const uint32_t empty = bar(m.kv_empty[stage]), done = bar(m.pv_done[j & 1]);
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < kTokens / 16; ++k)
#pragma unroll
            for (int c = 0; c < L::kColumns / 128; ++c)  // 128 of each CTA's columns
              ptx::mma_f16_ss_pair(
                  tmem + c * 128, ptx::desc_kmajor_sw128(weights + k * 32),
                  ptx::desc_mnmajor_sw128(values + (k / 2 * L::kHalf + 2 * c) * kBlockBytes +
                                              (k % 2) * 2048,
                                          kBlockBytes),
                  kOutputs, k > 0 ? 1u : add);
          ptx::mma_commit_pair(empty);
          ptx::mma_commit_pair(done);
        }
        __syncwarp();
      }
    }
    if (rank == 0 && ptx::elect_one()) ptx::mma_commit_pair(bar(m.drained[1]));
  } else if (warp == 2) {
    // ---------------------------------------------------------- keys' mender
    begin();
    // A draft with a non-finite number in its latent gets NaN for a score from
    // every row: an infinity alone could come out as a weight of zero.
    int r = 0, j = 0;
    bool ok = true;
    while (ok && next_segment(m.lists, p, cluster, walk, seg)) {
      for (int kv = seg.kv0 - 2; kv < seg.kv1; ++kv, ++r) {  // two of queries first
        ok = __all_sync(~0u, wait(m.kv_full[r % kStages], r / kStages));
        if (!ok) break;
        if (kv < seg.kv0) continue;
        if (special(seg, kv)) {
          uint8_t* keys = smem + r % kStages * L::kPlaceBytes;
          const int at = kv * kTokens + static_cast<int>(rank) * kCtaTokens;
          const int n0 = max(seg.context - at, 0), n1 = min(seg.length - at, kCtaTokens);
          // A token's 128-byte rows hold their 16-byte chunks in swizzled order,
          // which a search does not mind.
          for (int n = n0; n < n1; ++n) {
            bool finite = true;
#pragma unroll
            for (int i = 0; i < L::kBlocks * 8; i += 32)
              finite = finite && finite_bf16(*reinterpret_cast<const uint4*>(
                                     keys + (i + lane) / 8 * kBlockBytes + n * 128 + lane % 8 * 16));
            if (!__all_sync(~0u, finite) && lane == 0)
              *reinterpret_cast<uint16_t*>(keys + n * 128) = 0x7FC0u;
          }
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(first_cta(m.k_ready[j % kStages]));
        ++j;
      }
    }
    // The join may come: it reads this kernel's inputs, which are past the wait.
    // (With the first tiles it would take issue slots from them.)
    ptx::launch_dependents();
  } else if (warp == kValueMender) {
    // -------------------------------------------------------- values' mender
    begin();
    // Zeros for the tokens past the length and for drafts that are not finite:
    // rows that do not see them give them weights of zero.
    int r = 0, j = 0;
    bool ok = true;
    while (ok && next_segment(m.lists, p, cluster, walk, seg)) {
      r += 2;
      for (int kv = seg.kv0; kv < seg.kv1; ++kv, ++r, ++j) {
        ok = __all_sync(~0u, wait(m.v_full[j % kStages], j / kStages));
        if (!ok) break;
        if (special(seg, kv)) {
          wait(m.kv_full[r % kStages], r / kStages);  // (over since the keys' product)
          uint8_t* values = smem + r % kStages * L::kPlaceBytes;
          const int n0 = max(seg.context - kv * kTokens, 0);
          const int n1 = min(seg.length - kv * kTokens, kTokens);
          auto row_of = [&](int n) {
            return values + n / kCtaTokens * L::kHalf * kBlockBytes + n % kCtaTokens * 128;
          };
          uint64_t fill = 0;
          for (int n = n0; n < n1; ++n) {
            bool finite = true;
            if (lane < L::kHalf * 8)
              finite = finite_bf16(*reinterpret_cast<const uint4*>(
                  row_of(n) + lane / 8 * kBlockBytes + lane % 8 * 16));
            if (!__all_sync(~0u, finite)) fill |= 1ull << n;
          }
          // Boxes past the length came as zeros; the rest of the last one is
          // filled here.
          fill |= low_ones((n1 + ap.box - 1) & -ap.box) & ~low_ones(n1);
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (int n = lane / 8; n < kTokens; n += 4) {  // 8 lanes a token's row of 128 bytes
            if (!(fill >> n & 1)) continue;
#pragma unroll
            for (int block = 0; block < L::kHalf; ++block)
              *reinterpret_cast<uint4*>(row_of(n) + block * kBlockBytes + lane % 8 * 16) = zero;
          }
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(first_cta(m.v_ready[j % kStages]));
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    begin();
    const int group = (warp - kSoftmaxWarp) / 4;  // takes the tiles of this parity
    const int quarter = warp & 3;  // the 32 tensor-memory lanes this warp reaches
    // Quarters 0 and 1 hold the rows' scores of the first half of a tile's
    // tokens and the outputs' first half of the columns, 2 and 3 the second.
    const int half = quarter / 2, row = quarter % 2 * 32 + lane;
    const int place_of_row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t score = lanes + L::kS + group * kCtaTokens;
    // A row of weights is one 128-byte swizzled row, this thread's tokens half
    // of its chunks.
    uint8_t* weights = smem + L::kP + group * kWeightBytes + row * 128;
    uint32_t decisions = 0;  // tiles of this quarter's rows, of both groups
    int g = 0;               // token tiles before the segment
    int r = 0;               // places of the ring before its first token tile
    // The outputs of tile j are added.  A parity tells a phase from the next
    // alone: a group waits for its own tile j - 2 before it gives tile j's weights
    // away, so neither group's barrier is ever more than a phase ahead of a wait
    // (products, and their commits, are done in order).
    auto added = [&](int j) { wait(m.pv_done[j & 1], j >> 1); };
    auto all_added = [&](int tiles) {
      if (tiles > 1 && ((g + tiles) & 1) == group) added(g + tiles - 2);
      added(g + tiles - 1);
    };
    for (uint32_t segments = 0; next_segment(m.lists, p, cluster, walk, seg); ++segments) {
      const int tile_row = static_cast<int>(rank) * kCtaRows + row;
      const size_t q_row = static_cast<size_t>(seg.begin) * p.heads + seg.row0 + tile_row;
      const bool mine = tile_row < seg.valid;
      const bool active = tile_row - lane < seg.valid;  // of the warp
      const int tiles = seg.kv1 - seg.kv0;
      const int i0 = (g & 1) != group;  // this group's first tile
      // Queries, from the ring into tensor memory, half of the blocks a group.
      wait(m.kv_full[r % kStages], r / kStages);
      wait(m.kv_full[(r + 1) % kStages], (r + 1) / kStages);
      wait(m.q_full, segments);
      if (active) {
        const uint8_t* src = smem + (r + group) % kStages * L::kPlaceBytes + row * 128;
#pragma unroll
        for (int block = 0; block < L::kTmemBlocks / 2; ++block) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + block * kQBlockBytes +
                                                            ((i ^ (row & 7)) * 16));
            v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
          }
          ptx::tmem_st_32x32b_x32(lanes + L::kQ + (group * (L::kTmemBlocks / 2) + block) * 32, v);
        }
        ptx::tmem_wait_st();
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote(first_cta(m.q_ready));
      r += 2;
      if (!active) {
        for (int i = i0; i < tiles; i += 2) {
          wait(m.s_full[group], (g + i) >> 1);
          // (The scores two tiles on may come before this tile's weights: no
          // second arrival at one phase.)
          if (i >= 2) added(g + i - 2);
          if (lane == 0) {
            ptx::mbar_arrive_remote(first_cta(m.s_free[group]));
            ptx::mbar_arrive_remote(first_cta(m.p_full[group]));
          }
        }
        // Not on to the next segment before this one is done.
        all_added(tiles);
        g += tiles;
        r += tiles;
        continue;
      }
      // What this row sees of the drafts.
      const int t = (seg.row0 + tile_row) / p.heads;
      const uint64_t tree =
          p.tree != nullptr && mine ? static_cast<uint64_t>(p.tree[seg.begin + t]) : 0;
      // After this group's last tile: the reference, and the sum of this
      // thread's tokens under it.
      float base = -INFINITY, total = 0.0f;

      for (int i = i0; i < tiles; i += 2) {
        const int kv = seg.kv0 + i, j = g + i;
        const uint32_t decision = decisions + i;
        wait(m.s_full[group], j >> 1);
        ptx::tc_fence_after();
        uint32_t raw[32];
        ptx::tmem_ld_32x32b_x32(score, raw);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(first_cta(m.s_free[group]));
        float z[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) z[c] = __uint_as_float(raw[c]);
        bool any = true;  // of this thread's tokens is visible
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
          const uint32_t bits = static_cast<uint32_t>(sees >> (32 * half));
          any = bits != 0u;
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
        // The row's maximum, with the thread of its other tokens; the two
        // decide alike on the row's reference after this tile.
        float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        float* shared = m.tops[(j >> 1) & 1][group];
        shared[place_of_row] = top;
        asm volatile("bar.sync %0, 64;" ::"r"(3 + group * 2 + quarter % 2) : "memory");
        top = fmaxf(top, shared[place_of_row ^ 64]);
        float before = -INFINITY;
        if (i > 0) {
          wait(m.decided[(decision - 1) & 1][quarter], (decision - 1) >> 1);
          before = m.reference[(decision - 1) & 1][place_of_row];
        }
        const float now = (top - before) * p.scale_log2 > kLazy ? top : before;
        m.reference[decision & 1][place_of_row] = now;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(m.decided[decision & 1][quarter]));
        total *= shift_factor(base, now, p.scale_log2);
        base = now;
        const float sub = now == -INFINITY ? 0.0f : now;
        uint32_t w[16];
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        // (The reference in the scores' own units, subtracted before the scale: a
        // fused z scale - reference would leave of a great score what the
        // rounding of its product with the scale has left out, past 2^31 more
        // than the exponential takes.)
        const float2 by = make_float2(p.scale_log2, p.scale_log2), less = make_float2(-sub, -sub);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 x = mul2(add2(make_float2(z[2 * c], z[2 * c + 1]), less), by);
          w[c] = pack_bf16(exp2_approx(x.x), exp2_approx(x.y));
          sum[c % 2] = add2(sum[c % 2], make_float2(__uint_as_float(w[c] << 16),
                                                    __uint_as_float(w[c] & 0xFFFF0000u)));
        }
        sum[0] = add2(sum[0], sum[1]);
        total += sum[0].x + sum[0].y;
        if (now == -INFINITY && any && total == 0.0f) total = kAllInfinite;
        if (i >= 2) added(j - 2);  // this group's last weights are read
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(weights + (((half * 4 + c) ^ (row & 7)) * 16)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        if (i > 0 && __any_sync(~0u, now != before)) {
          // The outputs so far, once the tile before has been added.
          const float f = shift_factor(before, now, p.scale_log2);
          added(j - 1);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < L::kColumns; c += 32) {
            ptx::tmem_ld_32x32b_x32(lanes + c, raw);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 32; ++q) raw[q] = __float_as_uint(__uint_as_float(raw[q]) * f);
            ptx::tmem_st_32x32b_x32(lanes + c, raw);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(first_cta(m.p_full[group]));
      }

      // The row tile's outputs: the last tile is decided, and added.
      const uint32_t last = decisions + tiles - 1;
      decisions += tiles;
      wait(m.decided[last & 1][quarter], last >> 1);
      const float now = m.reference[last & 1][place_of_row];
      m.sums[group * 2 + half][row] = total * shift_factor(base, now, p.scale_log2);
      asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter % 2) : "memory");
      total = (m.sums[0][row] + m.sums[1][row]) + (m.sums[2][row] + m.sums[3][row]);
      all_added(tiles);
      ptx::tc_fence_after();
      const bool whole = seg.kv0 == 0 && seg.kv1 == seg.kv_tiles;
      const bool sectors = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
      const int lane_column = group * (L::kColumns / 2);
      const int column0 = half * L::kColumns + lane_column;
      const float inverse = inverse_of(total);
      if (!whole && half == 0 && group == 0 && mine)
        ap.stats[seg.slot * kTileRows + tile_row] = make_float2(now, total);
#pragma unroll 1
      for (int c = 0; c < L::kColumns / 2; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(lanes + lane_column + c, v);
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
            // A sector at once where the output begins on one (rows and columns
            // keep to it), which the C interface does not ask for.
            if (sectors) {
              ptx::st_v8(out + 16 * i, w);
            } else {
              uint4* chunk = reinterpret_cast<uint4*>(out + 16 * i);
              chunk[0] = make_uint4(w[0], w[1], w[2], w[3]);
              chunk[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        } else {
          float4* part = ap.partial +
                         (static_cast<size_t>(seg.slot) * (kLatent / 4) + (column0 + c) / 4) *
                             kTileRows +
                         tile_row;
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
  // Nothing runs on when tensor memory is freed, and no CTA leaves while its peer
  // may address it: each waits here for the issuers' last commits, which arrive
  // on both CTAs' barriers and are not shown to have reached the second one by
  // what the first one sees; every other arrival from the peer a role has waited
  // for.  (Nothing is handed over by the cluster's barrier: a release would wait
  // for the outputs' stores, 0.5 us.)
  if (warp == 1) {
    ptx::mbar_wait(bar(m.drained[0]), 0, kWaitLimitNs);
    ptx::mbar_wait(bar(m.drained[1]), 0, kWaitLimitNs);
  }
  __syncwarp();
  ptx::cluster_sync_relaxed();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Joins the partial outputs of the row tiles that several clusters shared, in
// the order of their tokens.  An item is a row tile's 8 columns, a thread a row
// by 4 of them.
constexpr int kJoinThreads = 256;
constexpr int kJoinColumns = kJoinThreads / kTileRows * 4;
template <int kLatent>
__global__ void __launch_bounds__(kJoinThreads, 3)
    join_kernel(const __grid_constant__ AttendParams ap) {
  ptx::launch_dependents();
  const LatentParams& p = ap.in;
  const int row = threadIdx.x % kTileRows;
  constexpr int kItems = kLatent / kJoinColumns;  // of a row tile
  ptx::grid_dependency_wait();
  // The cut row tiles, at most one a cluster, a lane each of 32 clusters.
  constexpr int kWords = (kMaxClusters + 31) / 32;
  Cut mine[kWords];
  uint32_t there[kWords];
  int cuts = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int c = w * 32 + threadIdx.x % 32;
    mine[w] = c < ap.clusters ? ap.cuts[c] : Cut{0, 0, 0, 0};
    there[w] = __ballot_sync(~0u, mine[w].rows > 0);
    cuts += __popc(there[w]);
  }
  for (int item = blockIdx.x; item < cuts * kItems; item += gridDim.x) {
    int n = item / kItems;
    Cut cut{};
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      uint32_t left = there[w];
      if (n >= 0 && n < __popc(left)) {
        for (int k = 0; k < n; ++k) left &= left - 1u;
        const int from = __ffs(left) - 1;
        cut.slot = __shfl_sync(~0u, mine[w].slot, from);
        cut.last = __shfl_sync(~0u, mine[w].last, from);
        cut.row0 = __shfl_sync(~0u, mine[w].row0, from);
        cut.rows = __shfl_sync(~0u, mine[w].rows, from);
      }
      n -= __popc(there[w]);
    }
    if (row >= cut.rows) continue;
    const int column = item % kItems * kJoinColumns + threadIdx.x / kTileRows * 4;
    const int c0 = cut.slot / 2;
    // Ten clusters' loads at a time (76 clusters on 8 row tiles make 9 or 10
    // parts), under the largest reference so far.
    constexpr int kBatch = 10;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float top = -INFINITY, total = 0.0f;
    float4 sum = zero;
    for (int c = c0; c <= cut.last; c += kBatch) {
      float2 st[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        st[k] = make_float2(-INFINITY, 0.0f);
        v[k] = zero;
        if (c + k > cut.last) continue;
        const int slot = c + k == c0 ? cut.slot : 2 * (c + k);
        st[k] = ap.stats[slot * kTileRows + row];
        v[k] =
            ap.partial[(static_cast<size_t>(slot) * (kLatent / 4) + column / 4) * kTileRows + row];
      }
      float next = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) next = fmaxf(next, st[k].x);
      const float keep = shift_factor(top, next, p.scale_log2);
      top = next;
      total *= keep;
      sum = make_float4(sum.x * keep, sum.y * keep, sum.z * keep, sum.w * keep);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = shift_factor(st[k].x, top, p.scale_log2);
        total = fmaf(f, st[k].y, total);
        sum.x = fmaf(f, v[k].x, sum.x), sum.y = fmaf(f, v[k].y, sum.y);
        sum.z = fmaf(f, v[k].z, sum.z), sum.w = fmaf(f, v[k].w, sum.w);
      }
    }
    const float inverse = inverse_of(total);
    *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(cut.row0) + row) * kLatent + column) =
        make_uint2(pack_bf16(sum.x * inverse, sum.y * inverse),
                   pack_bf16(sum.z * inverse, sum.w * inverse));
  }
}

constexpr int kMaxDevicesTracked = 64;

template <int kLatent>
constexpr uint32_t smem_bytes() {
  static_assert(MXFP8_MAX_LATENT_ROWS <= 65535, "row numbers fit 16 bits");
  constexpr uint32_t kBytes = Shape<kLatent>::kMisc + sizeof(Misc<Shape<kLatent>::kStages>);
  static_assert(kBytes <= 232448, "shared memory of a CTA");
  // The pair allocates all of tensor memory, which waits for whoever holds some;
  // no CTA that in turn waits for another (the projection's clusters ask for a
  // third of an SM's shared memory) may be on its SM.
  static_assert(kBytes > 233472 / 3 * 2, "an SM to itself");
  return kBytes;
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

// The cache as [page][block of 64 columns][token][64].
CUresult encode_cache(CUtensorMap* map, const LatentParams& p, int latent, int box, int blocks) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t page =
      p.pages > 1 ? p.page_stride : static_cast<int64_t>(p.page_size) * p.token_stride;
  cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(p.page_size),
                        static_cast<cuuint64_t>(latent / 64 + 1), static_cast<cuuint64_t>(p.pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.token_stride) * 2, 128, page * 2};
  cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(blocks), 1};
  cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(p.cache), dims,
            strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// q [rows x heads][latent + 64].
CUresult encode_queries(CUtensorMap* map, const LatentParams& p, int latent) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return CUDA_ERROR_NOT_FOUND;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(latent + kRope),
                        static_cast<cuuint64_t>(p.rows) * p.heads};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(latent + kRope) * 2};
  cuuint32_t boxes[2] = {64, kCtaRows};
  cuuint32_t elem[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p.q), dims, strides,
            boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int kLatent>
cudaError_t launch_impl(const LatentParams& p, void* workspace, cudaStream_t stream) {
  AttendParams ap{};
  ap.in = p;
  cudaError_t e = resident_clusters<kLatent>(&ap.clusters);
  if (e != cudaSuccess) return e;
  ap.box = kCtaTokens;
  while (p.page_size % ap.box) ap.box /= 2;
  while (1 << ap.box_log2 < ap.box) ++ap.box_log2;
  ap.by_page = divisor_of(p.page_size);
  ap.by_clusters = divisor_of(ap.clusters);
  ap.partial = static_cast<float4*>(workspace);
  ap.stats = reinterpret_cast<float2*>(ap.partial + static_cast<size_t>(2) * kMaxClusters *
                                                        (kLatent / 4) * kTileRows);
  ap.cuts = reinterpret_cast<Cut*>(ap.stats + static_cast<size_t>(2) * kMaxClusters * kTileRows);
  AttendMaps maps;
  using L = Shape<kLatent>;
  const bool whole = ap.box == kCtaTokens;
  if (encode_cache(&maps.keys, p, kLatent, ap.box, whole ? L::kBlocks + 1 : 1) != CUDA_SUCCESS ||
      encode_cache(&maps.values, p, kLatent, ap.box, whole ? L::kHalf : 1) != CUDA_SUCCESS ||
      encode_queries(&maps.q, p, kLatent) != CUDA_SUCCESS)
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
  // Row tiles of all requests at most.  None is cut where each fits the shortest
  // run and there is a cluster for each.
  const int tiles = static_cast<int>(static_cast<int64_t>(p.rows) * p.heads / kTileRows) +
                    std::min(p.requests, p.rows);
  if (tiles == 0 || (tiles <= ap.clusters &&
                     static_cast<int64_t>(p.table_width) * p.page_size <= kMinRun * kTokens))
    return cudaSuccess;
  cfg.gridDim = dim3(static_cast<unsigned>(
      std::min(std::min(tiles, ap.clusters) * (kLatent / kJoinColumns), 8 * ap.clusters)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<kLatent>, ap);
}

}  // namespace

size_t latent_workspace_bytes(int latent) {
  return static_cast<size_t>(2) * kMaxClusters * kTileRows *
             (static_cast<size_t>(latent) * sizeof(float) + sizeof(float2)) +
         kMaxClusters * sizeof(Cut);
}

cudaError_t launch_latent_attend(const LatentParams& p, int latent, void* workspace,
                                 cudaStream_t stream) {
  return latent == 512 ? launch_impl<512>(p, workspace, stream)
                       : launch_impl<256>(p, workspace, stream);
}

}  // namespace mxfp8
