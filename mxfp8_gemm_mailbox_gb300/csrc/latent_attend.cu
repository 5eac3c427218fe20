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
// every token, as key and as value.  A token crosses from L2 once per cluster
// and each CTA multiplies only its own columns: its scores are partial sums,
// exchanged in FP32 through distributed shared memory and added (the same two
// numbers in both CTAs, so both derive the same softmax), then multiplied into
// the CTA's own output columns.
//
// Work: the (request, row tile, 64-token tile) triples form one list, cut into
// equal runs, one a cluster, so ragged lengths balance by themselves.  A row
// tile cut between clusters leaves FP32 partial outputs with their maxima and
// sums, which a second kernel joins in a fixed order.
//
// Warps of a CTA:
//   0      producer: TMA boxes of a token tile into a ring, one lane a box;
//   1      MMA issuer: scores of tile j + 1, then outputs of tile j;
//   2      mender of the tiles that reach the drafts or the length: zeroes the
//          tokens past the length and drafts that are not finite;
//   4-19   softmax, two groups of eight that take the tiles in turn, so one
//          group's exchange and exponentials run under the other's products:
//          thread = row (tensor-memory lane), two warps a row, 32 of the 64
//          tokens each.  The reference of a row's exponentials passes from
//          tile to tile, and so between the groups, through shared memory.
//
// Precision: scores, maxima, sums, outputs and partials FP32; the weights e_p
// are rounded to BF16, the MMA's operand type (2^-8 relative at most), and the
// normaliser sums the rounded ones, so the weights that are applied sum to 1.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kRope = 64;
constexpr int kTokens = 64;     // tokens in a tile
constexpr int kTileRows = 128;  // rows in a tile
constexpr int kAttendThreads = 640;
constexpr int kSoftmaxWarp = 4;
constexpr int kMaxRequests = MXFP8_MAX_REQUESTS;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
// A new maximum moves the reference of a row's exponentials only when it
// passes it by this many powers of two: the weights then stay below 2^8, far
// inside FP32 and BF16, and the outputs in tensor memory are seldom rescaled.
constexpr float kLazy = 8.0f;
constexpr uint32_t kAtomBytes = kTokens * 128;  // 64 tokens x 64 columns
constexpr uint32_t kRopeBytes = kTokens * 64;   // 64 tokens x 32 rotary columns
constexpr uint32_t kQRopeBytes = kTileRows * 64;
constexpr uint32_t kRecvBytes = kTileRows * kTokens * 4;

template <int kLatent>
struct Shape {
  static constexpr int kHalf = kLatent / 2;  // columns of a CTA
  static constexpr int kAtoms = kHalf / 64;
  static constexpr uint32_t kStageBytes = kAtoms * kAtomBytes + kRopeBytes;
  static constexpr int kStages = kLatent == 512 ? 4 : 6;
  // Tensor-memory columns: outputs, queries (two BF16 a column), two score
  // tiles (their weights overwrite them).
  static constexpr uint32_t kQ = kHalf;
  static constexpr uint32_t kS = kHalf + kHalf / 2;
  static constexpr uint32_t kRecv = kStages * kStageBytes;
  static constexpr uint32_t kQRope = kRecv + 2 * kRecvBytes;
  static constexpr uint32_t kMisc = kQRope + kQRopeBytes;
  static_assert(kS + 2 * kTokens <= 512, "tensor memory");
};

struct Misc {
  uint64_t kv_full[6], kv_empty[6], kv_ready[6];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t recv_full[2][8], credit[2][8];  // [group][warp of the group]
  uint64_t decided[2][4];                  // [tile parity][lane quarter]
  uint64_t q_ready, drained;
  uint64_t bad[6];  // non-finite drafts of a stage's tile, one bit a token
  uint32_t tmem;
  int32_t abort;
  float top[2][2][kTileRows];       // [group][token half][row]
  float reference[2][kTileRows];    // [tile parity][row]
  float total[2][2][kTileRows];     // [group][token half][row]
  int64_t first[kMaxRequests + 1];  // tiles before each request
  int32_t length[kMaxRequests];
  uint16_t begin[kMaxRequests];     // rows are at most MXFP8_MAX_LATENT_ROWS
  uint16_t drafts[kMaxRequests];
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
  r.drafts = max(min(end, p.rows) - r.begin, 0);
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
// Tiles of a cluster's run.
__device__ __forceinline__ int64_t run_length(int64_t tiles, int clusters) {
  return max(static_cast<int64_t>(1), (tiles + clusters - 1) / clusters);
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One row tile's run of token tiles inside a cluster's run.
struct Segment {
  int b, kv0, kv1, kv_tiles;
  int length, context, drafts, begin;
  int row0;   // first row of the tile within the request (drafts x heads rows)
  int valid;  // rows of the tile, at most 128
};
struct Walk {
  int64_t at, end;
  int b;
};
__device__ __forceinline__ bool next_segment(const Misc& m, const LatentParams& p, Walk& w,
                                             Segment& s) {
  if (w.at >= w.end) return false;
  while (w.at >= m.first[w.b + 1]) ++w.b;
  s.b = w.b;
  s.length = m.length[w.b];
  s.begin = m.begin[w.b];
  s.drafts = m.drafts[w.b];
  s.context = max(s.length - s.drafts, 0);
  s.kv_tiles = token_tiles(s.length);
  const int64_t local = w.at - m.first[w.b];
  const int tile = static_cast<int>(local / s.kv_tiles);
  s.kv0 = static_cast<int>(local % s.kv_tiles);
  s.kv1 = static_cast<int>(min(static_cast<int64_t>(s.kv_tiles), s.kv0 + (w.end - w.at)));
  s.row0 = tile * kTileRows;
  s.valid = min(kTileRows, s.drafts * p.heads - s.row0);
  w.at += s.kv1 - s.kv0;
  return true;
}
// Whether a token tile reaches the drafts or the length.
__device__ __forceinline__ bool special(const Segment& s, int kv) {
  return (kv + 1) * kTokens > s.context;
}

// Bounded waits of a warp's converged lanes.  One that runs out sets `abort`,
// after which every wait of the CTA returns at once: the roles then run their
// loops out on whatever the buffers hold, so that no barrier is left short of
// an arrival, and the kernel ends with its flag set.
struct Waiter {
  int32_t* abort;
  int32_t* flags;
  __device__ __forceinline__ bool operator()(const uint64_t& b, uint32_t parity) const {
    const uint32_t bar = ptx::smem_addr(&b);
    return __all_sync(~0u, ptx::mbar_try_wait(bar, parity & 1u)) || slow(bar, parity & 1u, false);
  }
  // With acquire over the cluster, for what a peer CTA signals.
  __device__ __forceinline__ bool cluster(const uint64_t& b, uint32_t parity) const {
    const uint32_t bar = ptx::smem_addr(&b);
    return __all_sync(~0u, ptx::mbar_try_wait_cluster(bar, parity & 1u)) ||
           slow(bar, parity & 1u, true);
  }
  __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity, bool wide) const {
    const uint64_t start = ptx::globaltimer();
    for (;;) {
      if (__any_sync(~0u, *reinterpret_cast<volatile int32_t*>(abort) != 0)) return false;
      for (int i = 0; i < 32; ++i)
        if (__all_sync(~0u, wide ? ptx::mbar_try_wait_cluster(bar, parity)
                                 : ptx::mbar_try_wait(bar, parity)))
          return true;
      if (__any_sync(~0u, ptx::globaltimer() - start > kWaitLimitNs)) {
        *reinterpret_cast<volatile int32_t*>(abort) = 1;
        raise(flags, MXFP8_FLAG_GEMM_TIMEOUT);
        return false;
      }
    }
  }
};

struct AttendParams {
  LatentParams in;
  int32_t clusters;
  int32_t box;        // tokens of a TMA box: gcd(page_size, 64)
  float4* partial;    // [2 clusters][latent / 4][128 rows] x 4 columns
  float2* stats;      // [2 clusters][128 rows] (reference exponent, sum)
};

template <int kLatent>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmap_c,
                  const __grid_constant__ CUtensorMap tmap_r,
                  const __grid_constant__ AttendParams ap) {
  using L = Shape<kLatent>;
  constexpr int kWidth = kLatent + kRope;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = ptx::smem_addr(smem);
  Misc& m = *reinterpret_cast<Misc*>(smem + L::kMisc);
  const LatentParams& p = ap.in;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = ptx::cluster_ctarank();
  const int cluster = blockIdx.x / 2;
  auto bar = [&](const uint64_t& b) { return ptx::smem_addr(&b); };

  if (tid == 0) {
    ptx::prefetch_tensormap(&tmap_c);
    ptx::prefetch_tensormap(&tmap_r);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bar(m.kv_full[i]), 1);
      ptx::mbar_init(bar(m.kv_empty[i]), 2);  // the outputs' commit and the mender
      ptx::mbar_init(bar(m.kv_ready[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(m.s_full[i]), 1);
      ptx::mbar_init(bar(m.p_full[i]), 8);
      ptx::mbar_init(bar(m.pv_done[i]), 1);
      for (int w = 0; w < 4; ++w) ptx::mbar_init(bar(m.decided[i][w]), 2);
      for (int w = 0; w < 8; ++w) {
        ptx::mbar_init(bar(m.recv_full[i][w]), 1);
        ptx::mbar_init(bar(m.credit[i][w]), 1);
      }
    }
    ptx::mbar_init(bar(m.q_ready), 16);
    ptx::mbar_init(bar(m.drained), 1);
    m.abort = 0;
    ptx::fence_mbarrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(bar(reinterpret_cast<uint64_t&>(m.tmem)), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = m.tmem;
  if (tid == 0) ptx::launch_dependents();
  ptx::grid_dependency_wait();

  // Tiles before each request, by one warp.
  if (warp == 0) {
    int64_t before = 0;
    for (int base = 0; base < p.requests; base += 32) {
      const int b = base + lane;
      int64_t tiles = 0;
      if (b < p.requests) {
        const Request r = load_request(p, b);
        if (r.cut && blockIdx.x == 0) raise(p.flags, MXFP8_FLAG_BAD_INDEX);
        m.length[b] = r.length;
        m.begin[b] = static_cast<uint16_t>(r.begin);
        m.drafts[b] = static_cast<uint16_t>(r.drafts);
        tiles = static_cast<int64_t>(row_tiles(r.drafts, p.heads)) * token_tiles(r.length);
      }
      for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(~0u, tiles, o);
        if (lane >= o) tiles += v;
      }
      if (b < p.requests) m.first[b + 1] = before + tiles;
      before += __shfl_sync(~0u, tiles, 31);
    }
    if (lane == 0) m.first[0] = 0;
  }
  __syncthreads();
  const int64_t all = m.first[p.requests];
  const int64_t run = run_length(all, ap.clusters);
  const int64_t run_begin = min(all, cluster * run);
  Walk walk{run_begin, min(all, run_begin + run), 0};
  Segment seg{};
  const Waiter wait{&m.abort, p.flags};

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    // A lane a box (one thread's copies are served one after another); the
    // page of a lane's box is looked up one tile ahead.
    constexpr int kItems = (8 * (L::kAtoms + 1) + 31) / 32;  // of a lane, boxes of 8 tokens
    auto page_of = [&](int kv, int i) {
      const int token = kv * kTokens + i / (L::kAtoms + 1) * ap.box;
      if (token >= seg.length) return 0;
      const int page = p.table[static_cast<size_t>(seg.b) * p.table_width + token / p.page_size];
      if (page >= 0 && page < p.pages) return page;
      raise(p.flags, MXFP8_FLAG_BAD_INDEX);
      return p.pages;  // past the tensor: the copy fills zeros
    };
    const int boxes_per_tile = kTokens / ap.box;
    int g = 0;
    bool ok = true;
    while (ok && next_segment(m, p, walk, seg)) {
      int page[kItems];
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = lane + 32 * k;
        page[k] = i < boxes_per_tile * (L::kAtoms + 1) ? page_of(seg.kv0, i) : 0;
      }
      for (int kv = seg.kv0; kv < seg.kv1; ++kv, ++g) {
        const int stage = g % kStages;
        const uint32_t use = static_cast<uint32_t>(g / kStages);
        int next[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          const int i = lane + 32 * k;
          next[k] = kv + 1 < seg.kv1 && i < boxes_per_tile * (L::kAtoms + 1) ? page_of(kv + 1, i)
                                                                             : 0;
        }
        if (g >= kStages) ok = wait(m.kv_empty[stage], use - 1);
        if (!ok) break;
        const int boxes = min(boxes_per_tile, (seg.length - kv * kTokens + ap.box - 1) / ap.box);
        const uint32_t full = bar(m.kv_full[stage]);
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * ap.box) *
                                               (L::kHalf * 2u + 64u));
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          const int i = lane + 32 * k;
          if (i >= boxes * (L::kAtoms + 1)) continue;
          const int box = i / (L::kAtoms + 1), atom = i % (L::kAtoms + 1);
          const int at = (kv * kTokens + box * ap.box) % p.page_size;
          const uint32_t dst = sbase + stage * L::kStageBytes;
          if (atom < L::kAtoms)
            ptx::tma_load_3d(dst + atom * kAtomBytes + box * ap.box * 128, &tmap_c,
                             static_cast<int>(rank) * L::kHalf + atom * 64, at, page[k], full,
                             ptx::policy_evict_last());
          else
            ptx::tma_load_3d(dst + L::kAtoms * kAtomBytes + box * ap.box * 64, &tmap_r,
                             static_cast<int>(rank) * 32, at, page[k], full,
                             ptx::policy_evict_last());
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kItems; ++k) page[k] = next[k];
      }
    }
    // Copies in flight land before the CTA leaves (they have, unless a wait
    // ran out).
    for (int i = max(0, g - kStages); i < g; ++i)
      ptx::mbar_wait(bar(m.kv_full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u,
                     kWaitLimitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The warp stays converged and one elected lane issues: 32 clocks a
    // 128 x 64 x 16 product with the queries in tensor memory, the rate of the
    // tensor core; from a branch on the lane number it took 46.
    constexpr uint32_t kScores = ptx::idesc_bf16(kTokens, false);
    constexpr uint32_t kOutputs = ptx::idesc_bf16(L::kHalf, true);
    const uint32_t q_rope = sbase + L::kQRope;
    int g = 0;
    uint32_t segments = 0;
    bool ok = true;
    auto scores = [&](int j, int kv) {
      const int stage = j % kStages;
      if (!wait(special(seg, kv) ? m.kv_ready[stage] : m.kv_full[stage], j / kStages)) return false;
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
      return true;
    };
    while (ok && next_segment(m, p, walk, seg)) {
      ok = wait(m.q_ready, segments++);
      if (!ok) break;
      ptx::tc_fence_after();
      ok = scores(g, seg.kv0);
      if (ok && seg.kv0 + 1 < seg.kv1) ok = scores(g + 1, seg.kv0 + 1);
      for (int kv = seg.kv0; ok && kv < seg.kv1; ++kv, ++g) {
        ok = wait(m.p_full[g & 1], g >> 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const int stage = g % kStages;
        const uint32_t kvb = sbase + stage * L::kStageBytes;
        const uint32_t a = tmem + L::kS + (g & 1) * kTokens;
        const uint32_t add = kv > seg.kv0;
        const uint32_t empty = bar(m.kv_empty[stage]), done = bar(m.pv_done[g & 1]);
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < kTokens / 16; ++k)
            ptx::mma_f16_ts(tmem, a + k * 8, ptx::desc_mnmajor_sw128(kvb + k * 2048, kAtomBytes),
                            kOutputs, k > 0 ? 1u : add);
          ptx::mma_commit(empty);
          ptx::mma_commit(done);
        }
        __syncwarp();
        // Its weights read, the score buffer takes the tile after the next.
        if (kv + 2 < seg.kv1) ok = scores(g + 2, kv + 2);
      }
    }
    // Nothing runs on when tensor memory is freed.
    if (ptx::elect_one()) ptx::mma_commit(bar(m.drained));
    __syncwarp();
    ptx::mbar_wait(bar(m.drained), 0, kWaitLimitNs);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- mender
    int g = 0;
    bool ok = true;
    while (ok && next_segment(m, p, walk, seg)) {
      for (int kv = seg.kv0; ok && kv < seg.kv1; ++kv, ++g) {
        const int stage = g % kStages;
        ok = wait(m.kv_full[stage], g / kStages);
        if (!ok) break;
        if (special(seg, kv)) {
          uint8_t* kvp = smem + stage * L::kStageBytes;
          const int n0 = max(seg.context - kv * kTokens, 0);
          const int n1 = min(seg.length - kv * kTokens, kTokens);
          // A token's 128-byte rows hold their 16-byte chunks in swizzled order,
          // which neither a search nor a fill minds.
          uint64_t bad = 0;
          for (int n = n0; n < n1; ++n) {
            bool finite = true;
            for (int i = lane; i < L::kAtoms * 8; i += 32) {
              const uint4 v = *reinterpret_cast<const uint4*>(kvp + (i / 8) * kAtomBytes +
                                                              n * 128 + (i % 8) * 16);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                finite = finite && (w[q] & 0x7F80u) != 0x7F80u &&
                         (w[q] & 0x7F800000u) != 0x7F800000u;
            }
            if (!__all_sync(~0u, finite)) bad |= 1ull << n;
          }
          for (int n = n0; n < kTokens; ++n) {
            if (n < n1 && !(bad >> n & 1)) continue;
            for (int i = lane; i < L::kAtoms * 8 + 4; i += 32) {
              uint8_t* at = i < L::kAtoms * 8
                                ? kvp + (i / 8) * kAtomBytes + n * 128 + (i % 8) * 16
                                : kvp + L::kAtoms * kAtomBytes + n * 64 + (i - L::kAtoms * 8) * 16;
              *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
            }
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
    const int group = (warp - kSoftmaxWarp) / 8;  // takes the tiles of this parity
    const int sw = (warp - kSoftmaxWarp) % 8;
    const int quarter = warp & 3;  // the 32 tensor-memory lanes this warp reaches
    const int half = sw >> 2;      // its 32 of a tile's 64 tokens
    const int part = group * 2 + half;  // its quarter of the columns, in and out
    const int row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t score = lanes + L::kS + group * kTokens;
    const uint32_t peer = rank ^ 1u;
    const uint32_t recv_offset = L::kRecv + group * kRecvBytes + static_cast<uint32_t>(sw) * 4096u;
    const uint32_t recv_bar = bar(m.recv_full[group][sw]);
    const uint32_t to = ptx::map_to_rank(sbase + recv_offset + lane * 16u, peer);
    const uint32_t to_bar = ptx::map_to_rank(recv_bar, peer);
    const uint32_t credit_bar = ptx::map_to_rank(bar(m.credit[group][sw]), peer);
    const float4* recv = reinterpret_cast<const float4*>(smem + recv_offset) + lane;
    constexpr int kPart = L::kHalf / 4;
    uint32_t exchanges = 0;  // tiles this warp exchanged
    uint32_t decisions = 0;  // tiles this quarter's rows took part in, of both groups
    int g = 0;               // token tiles before the segment
    for (uint32_t segments = 0; next_segment(m, p, walk, seg);
         g += seg.kv1 - seg.kv0, ++segments) {
      const size_t q_row = static_cast<size_t>(seg.begin) * p.heads + seg.row0 + row;
      const bool mine = row < seg.valid;
      const bool active = quarter * 32 < seg.valid;  // of the warp
      // Queries: this CTA's columns into tensor memory, the rotary part into
      // shared memory (64-byte swizzle); rows past the tile are zero.
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + q_row * kWidth);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint32_t v[kPart / 2];
#pragma unroll
        for (int i = 0; i < kPart / 8; ++i) {
          const uint4 x = mine ? src[(rank * L::kHalf + part * kPart) / 8 + i] : zero;
          v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        }
        if constexpr (kPart == 64)
          ptx::tmem_st_32x32b_x32(lanes + L::kQ + part * (kPart / 2), v);
        else
          ptx::tmem_st_32x32b_x16(lanes + L::kQ + part * (kPart / 2), v);
        const uint4 x = mine ? src[kLatent / 8 + rank * 4 + part] : zero;
        *reinterpret_cast<uint4*>(smem + L::kQRope + row * 64 + ((part ^ ((row >> 1) & 3)) * 16)) =
            x;
        ptx::tmem_wait_st();
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(m.q_ready));
      }
      const int tiles = seg.kv1 - seg.kv0;
      if (!active) {
        for (int i = (g & 1) != group; i < tiles; i += 2) {
          wait(m.s_full[group], (g + i) >> 1);
          if (lane == 0) ptx::mbar_arrive(bar(m.p_full[group]));
        }
        // Not on to the next segment's queries before every warp's of this one.
        wait(m.q_ready, segments);
        continue;
      }
      // What this row sees of the drafts.
      const int t = (seg.row0 + row) / p.heads;
      const uint64_t tree =
          p.tree != nullptr && mine ? static_cast<uint64_t>(p.tree[seg.begin + t]) : 0;
      float reference = -INFINITY, total = 0.0f;  // of this warp's tiles

      for (int i = (g & 1) != group; i < tiles; i += 2, ++exchanges) {
        const int kv = seg.kv0 + i;
        const uint32_t decision = decisions + i;
        // This CTA's partial scores, sent to the peer and joined with its own.
        wait(m.s_full[group], (g + i) >> 1);
        ptx::tc_fence_after();
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(score + half * 32, v);
        ptx::tmem_wait_ld();
        if (special(seg, kv)) {
          const int stage = (g + i) % kStages;
          wait(m.kv_ready[stage], (g + i) / kStages);
          const uint32_t bad = static_cast<uint32_t>(m.bad[stage] >> (32 * half));
          if (bad != 0u)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (bad >> c & 1u) v[c] = 0x7FC00000u;
        }
        if (exchanges > 0) wait.cluster(m.credit[group][sw], exchanges - 1);
        if (lane == 0) ptx::mbar_arrive_expect_tx(recv_bar, 4096);
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          ptx::st_async_remote_v4(
              to + c * 512, make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]), to_bar);
        wait.cluster(m.recv_full[group][sw], exchanges);
        float z[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 x = recv[c * 32];
          z[4 * c] = __uint_as_float(v[4 * c]) + x.x;
          z[4 * c + 1] = __uint_as_float(v[4 * c + 1]) + x.y;
          z[4 * c + 2] = __uint_as_float(v[4 * c + 2]) + x.z;
          z[4 * c + 3] = __uint_as_float(v[4 * c + 3]) + x.w;
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
          const uint32_t bits = static_cast<uint32_t>(sees >> (32 * half));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(bits >> c & 1u)) z[c] = -INFINITY;
        }
        float top = z[0];
#pragma unroll
        for (int c = 1; c < 32; ++c) top = fmaxf(top, z[c]);
        m.top[group][half][row] = top;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + group * 4 + quarter) : "memory");
        top = fmaxf(top, m.top[group][half ^ 1][row]) * p.scale_log2;

        // The reference after the tile before this one, moved if the new
        // maximum passes it by more than kLazy.
        float now = -INFINITY;
        if (i > 0) {
          wait(m.decided[(decision - 1) & 1][quarter], (decision - 1) >> 1);
          now = m.reference[(decision - 1) & 1][row];
        }
        const bool move = top > now + kLazy;
        if (i > 0 && __any_sync(~0u, move)) {
          // The outputs so far, once the previous tile's have been added.
          const float f = move ? exp2_approx(now - top) : 1.0f;
          wait(m.pv_done[group ^ 1], (g + i - 1) >> 1);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < L::kHalf / 2; c += 32) {
            ptx::tmem_ld_32x32b_x32(lanes + half * (L::kHalf / 2) + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * f);
            ptx::tmem_st_32x32b_x32(lanes + half * (L::kHalf / 2) + c, v);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
        }
        if (move) now = top;
        if (half == 0) m.reference[decision & 1][row] = now;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(m.decided[decision & 1][quarter]));
        if (now != reference) {
          total *= exp2_approx(reference - now);
          reference = now;
        }
        const float base = now == -INFINITY ? 0.0f : now;
        uint32_t w[16];
        float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          w[c] = pack_bf16(exp2_approx(fmaf(z[2 * c], p.scale_log2, -base)),
                           exp2_approx(fmaf(z[2 * c + 1], p.scale_log2, -base)));
          sum0 += __uint_as_float(w[c] << 16);
          sum1 += __uint_as_float(w[c] & 0xFFFF0000u);
        }
        total += sum0 + sum1;
        ptx::tmem_st_32x32b_x16(score + half * 16, w);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(m.p_full[group]));
          // The peer may overwrite the receive buffer.  (Last: a release over
          // the cluster waits for this thread's own remote stores.)
          ptx::mbar_arrive_remote(credit_bar);
        }
      }

      // The row tile's outputs: the last tile's have been added, and the sums of
      // the row's four warps join under the last reference.
      const uint32_t last = decisions + tiles - 1;
      decisions += tiles;
      // In this order: once the last tile is decided its outputs' barrier is at
      // most one phase ahead of a look at its parity.
      wait(m.decided[last & 1][quarter], last >> 1);
      wait(m.pv_done[(g + tiles - 1) & 1], (g + tiles - 1) >> 1);
      ptx::tc_fence_after();
      const float now = m.reference[last & 1][row];
      if (now != reference) total *= exp2_approx(reference - now);
      m.total[group][half][row] = total;
      asm volatile("bar.sync %0, 128;" ::"r"(9 + quarter) : "memory");
      total = (m.total[0][0][row] + m.total[0][1][row]) + (m.total[1][0][row] + m.total[1][1][row]);
      const bool whole = seg.kv0 == 0 && seg.kv1 == seg.kv_tiles;
      const int column0 = static_cast<int>(rank) * L::kHalf + part * kPart;
      const int slot = 2 * cluster + (walk.at - tiles == run_begin ? 0 : 1);
      const float inverse = total == 0.0f ? 0.0f : 1.0f / total;
      if (!whole && rank == 0 && part == 0 && mine)
        ap.stats[slot * kTileRows + row] = make_float2(now, total);
#pragma unroll 1
      for (int c = 0; c < kPart; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(lanes + part * kPart + c, v);
        ptx::tmem_wait_ld();
        if (!mine) continue;
        if (whole) {
          uint4* out = reinterpret_cast<uint4*>(p.out + q_row * kLatent + column0 + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = pack_bf16(__uint_as_float(v[8 * i + 2 * q]) * inverse,
                               __uint_as_float(v[8 * i + 2 * q + 1]) * inverse);
            out[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* to_part = ap.partial +
                            (static_cast<size_t>(slot) * (kLatent / 4) + (column0 + c) / 4) *
                                kTileRows +
                            row;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to_part[i * kTileRows] =
                make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                            __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        }
      }
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
  ptx::grid_dependency_wait();
  const LatentParams& p = ap.in;
  const int row = threadIdx.x % kTileRows;
  const int column = blockIdx.y * 8 + (threadIdx.x / kTileRows) * 4;
  int64_t all = 0, begin = 0, end = 0;
  int tiles = 0, covered0 = p.rows, covered1 = p.rows;
  size_t out_row = 0;
  bool mine = false, found = false;
  for (int b = 0; b < p.requests; ++b) {
    const Request r = load_request(p, b);
    if (b == 0) covered0 = r.begin;
    if (b == p.requests - 1) covered1 = r.begin + r.drafts;
    const int rt = row_tiles(r.drafts, p.heads), kt = token_tiles(r.length);
    const int tile = static_cast<int>(blockIdx.x) - tiles;
    if (tile >= 0 && tile < rt) {
      found = true;
      begin = all + static_cast<int64_t>(tile) * kt;
      end = begin + kt;
      mine = tile * kTileRows + row < r.drafts * p.heads;
      out_row = static_cast<size_t>(r.begin) * p.heads + tile * kTileRows + row;
    }
    tiles += rt;
    all += static_cast<int64_t>(rt) * kt;
  }
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
  if (!found || !mine) return;
  if (begin == end) {
    write(out_row, zero);
    return;
  }
  const int64_t run = run_length(all, ap.clusters);
  const int c0 = static_cast<int>(begin / run), c1 = static_cast<int>((end - 1) / run);
  if (c0 == c1) return;  // one cluster wrote the whole
  auto slot_of = [&](int c) { return 2 * c + (c * run < begin ? 1 : 0); };
  float top = -INFINITY;
  for (int c = c0; c <= c1; ++c) top = fmaxf(top, ap.stats[slot_of(c) * kTileRows + row].x);
  if (top == -INFINITY) top = 0.0f;
  float4 sum = zero;
  float total = 0.0f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const int slot = slot_of(c);
    const float2 st = ap.stats[slot * kTileRows + row];
    const float4 v =
        ap.partial[(static_cast<size_t>(slot) * (kLatent / 4) + column / 4) * kTileRows + row];
    const float f = exp2_approx(st.x - top);
    total = fmaf(f, st.y, total);
    sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
    sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
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
  static_assert(Shape<kLatent>::kMisc + sizeof(Misc) + 1024 <= 232448, "shared memory of a CTA");
  return Shape<kLatent>::kMisc + sizeof(Misc) + 1024;
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
  CUtensorMap tmap_c, tmap_r;
  if (encode_cache(&tmap_c, p, 0, kLatent, ap.box, 64, CU_TENSOR_MAP_SWIZZLE_128B) !=
          CUDA_SUCCESS ||
      encode_cache(&tmap_r, p, kLatent, kRope, ap.box, 32, CU_TENSOR_MAP_SWIZZLE_64B) !=
          CUDA_SUCCESS)
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
  e = cudaLaunchKernelEx(&cfg, attend_kernel<kLatent>, tmap_c, tmap_r, ap);
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
         (static_cast<size_t>(latent) * sizeof(float) + sizeof(float2));
}

cudaError_t launch_latent_attend(const LatentParams& p, int latent, void* workspace,
                                 cudaStream_t stream) {
  return latent == 512 ? launch_impl<512>(p, workspace, stream)
                       : launch_impl<256>(p, workspace, stream);
}

}  // namespace mxfp8
