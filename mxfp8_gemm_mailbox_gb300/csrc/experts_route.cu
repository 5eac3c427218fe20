// Around the experts' products: the choice of each token's experts, the tokens
// in the experts' order, and the sum of what the experts gave.
//
// Route.  Token t's experts are those of its k largest logits, ties to the
// lowest index; its weights exp(z_e - z_max) over the sum of those (or of all).
// A slot is a row of the experts' products: slots are numbered by expert, then
// by token.  A logit of -infinity is not chosen: such an entry has no slot.
//
// Logits become integers of the same order with the index below them (32 bits for logits of
// 16, else 64), no two alike.  Up to eight choices: eight lanes take a token, each sorts its
// keys by eights and merges the larger eight of two lists until it has one, and three
// exchanges merge the lanes'; lane j then has the j-th choice.  Past eight a warp takes a
// token, each lane's keys sorted once; a step of the choice is a warp reduction over the
// lanes' first keys (for FP32 a second one, over the indexes of the lanes that have the
// largest), and the lane that gave it moves its keys up: 150 clocks each, so two tokens a
// warp go side by side.  (By such steps alone, 32 tokens, 128 experts, k 8 took 4.5 us in
// place of 2.6, 16384 tokens, 256 experts 18.2 in place of 12.5.)
//
// An expert appears once at most among a token's, so a block of tokens is, for each expert,
// a bit mask: its population is the block's count, and that of the bits below a token the
// token's place.  Nothing depends on the order of atomics.  One block does all of up to 32
// tokens; for more a second kernel gives the places, each block adding up the counts of
// those before it; past 64 blocks a kernel between the two adds them (63 blocks 6.9 us so,
// 6.6 without; 94 blocks 7.7 and 8.1).
//
// Bound by instructions where there are many tokens (a lane's compares and exchanges, which
// issue at half rate, are most of them) and by three launches that wait for one another:
// 16384 tokens, 256 experts, k 8 13.4 us (12.5 with the logits in L2; they are 1.2 us'
// reading; the kernels alone, cold: choice 8.1, sums 4.7, places 5.1); a token 2.8 us, 500
// tokens of 128 experts 4.6, 100000 31.
//
// Combine.  out[t] = add[t] + sum_j weight[t][j] y[slot[t][j]], in FP32, j
// ascending, rounded once; a thread has 8 numbers of a row, and its loads are
// all under way at once.  Bound by the memory: 4096 tokens, 8 rows of 4096 each, 47.6 us for
// 302 MB (6.3 TB/s); one token 1.9 us, the launch and two round trips.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
static_assert(kThreads == MXFP8_MAX_EXPERTS, "a thread an expert");

// Larger values have larger keys; +0 and -0 one; NaN the largest of all.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return ~0u;
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}
constexpr uint32_t kNothing = 0x007FFFFFu;  // order_key(-infinity)

// Two keys of 16 bits from two numbers of a 16-bit type, in order: adding zero makes
// +0 of -0 and one NaN, the largest, of all; then negative ones are turned over.
template <int kType>
__device__ __forceinline__ uint32_t short_keys(uint32_t w) {
  if constexpr (kType == MXFP8_BF16) {
    const __nv_bfloat162 v =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.0f));
    w = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __hadd2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(0.0f));
    w = *reinterpret_cast<const uint32_t*>(&v);
  }
  const uint32_t negative = w >> 15 & 0x00010001u;
  return w ^ (negative * 0xFFFFu | 0x80008000u);
}
template <int kType>
__device__ __forceinline__ float short_value(uint32_t key) {
  const uint32_t h = (key >> 15) ? key & 0x7FFFu : ~key & 0xFFFFu;
  if constexpr (kType == MXFP8_BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// A key and below it the index, smaller for a higher one.
template <int kType>
struct KeyOf {
  using T = uint32_t;
};
template <>
struct KeyOf<MXFP8_FP32> {
  using T = uint64_t;
};

// A key's logit, and whether that is -infinity (or the key none).
template <int kType>
__device__ __forceinline__ float value_of(typename KeyOf<kType>::T key) {
  if constexpr (kType == MXFP8_FP32)
    return key_value(static_cast<uint32_t>(key >> 32));
  else
    return short_value<kType>(key >> 16);
}
template <int kType>
__device__ __forceinline__ bool is_nothing(typename KeyOf<kType>::T key) {
  if constexpr (kType == MXFP8_FP32)
    return static_cast<uint32_t>(key >> 32) <= kNothing;
  else
    return key >> 16 <= (kType == MXFP8_BF16 ? 0x007Fu : 0x03FFu);
}

// Descending, by Batcher's odd-even merges.
template <int kEach, typename T>
__device__ __forceinline__ void sort_down(T (&k)[kEach]) {
#pragma unroll
  for (int p = 1; p < kEach; p *= 2)
#pragma unroll
    for (int q = p; q > 0; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < kEach; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (j + i + q < kEach && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
            const T a = k[j + i], b = k[j + i + q];
            k[j + i] = a > b ? a : b;
            k[j + i + q] = a > b ? b : a;
          }
}

// A lane's logits are neighbours in pairs.
template <int kType, int kEach>
__device__ __forceinline__ void load_keys(const RouteParams& p, int64_t t,
                                          typename KeyOf<kType>::T (&key)[kEach]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < kEach; i += 2) {
    const int e = 2 * lane + 32 * i;
    key[i] = key[i + 1] = 0u;
    if (e >= p.experts) continue;
    const bool both = e + 1 < p.experts;
    if constexpr (kType != MXFP8_FP32) {
      const uint16_t* const at = static_cast<const uint16_t*>(p.logits) + t * p.stride + e;
      const uint32_t w = p.pairs ? *reinterpret_cast<const uint32_t*>(at)
                                 : at[0] | (both ? static_cast<uint32_t>(at[1]) << 16 : 0u);
      const uint32_t keys = short_keys<kType>(w);
      key[i] = keys << 16 | (0xFFFFu - e);
      if (both) key[i + 1] = (keys & 0xFFFF0000u) | (0xFFFFu - (e + 1));
    } else {
      const float* const at = static_cast<const float*>(p.logits) + t * p.stride + e;
      key[i] = static_cast<uint64_t>(order_key(at[0])) << 32 | (0xFFFFu - e);
      if (both) key[i + 1] = static_cast<uint64_t>(order_key(at[1])) << 32 | (0xFFFFu - (e + 1));
    }
  }
}

// The experts and weights of kAtOnce tokens (bits bit, bit + kWarps of the block's masks),
// from their keys; the tokens' steps, 150 clocks each, do not wait for one another.
template <int kType, int kEach, int kAtOnce>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t0, int tokens, int bit,
                                       typename KeyOf<kType>::T (&key)[kAtOnce][kEach],
                                       uint32_t (*mask)[MXFP8_MAX_EXPERTS]) {
  constexpr bool kShort = kType != MXFP8_FP32;
  using Key = typename KeyOf<kType>::T;
  const int lane = threadIdx.x % 32;
  Key first[kAtOnce], mine[kAtOnce];  // lane j: the j-th chosen key
  float total[kAtOnce];
#pragma unroll
  for (int n = 0; n < kAtOnce; ++n) {
    sort_down(key[n]);
    first[n] = mine[n] = 0u;
    total[n] = 0.0f;
  }
  for (int j = 0; j < p.k; ++j) {
    Key top[kAtOnce];
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      if constexpr (kShort) {
        top[n] = __reduce_max_sync(~0u, key[n][0]);
      } else {
        const uint32_t high = __reduce_max_sync(~0u, static_cast<uint32_t>(key[n][0] >> 32));
        const uint32_t low =
            static_cast<uint32_t>(key[n][0] >> 32) == high ? key[n][0] & 0xFFFFu : 0u;
        top[n] = static_cast<uint64_t>(high) << 32 | __reduce_max_sync(~0u, low);
      }
    }
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const bool live = !is_nothing<kType>(top[n]);  // else -infinity from here on
      if (j == 0) {
        first[n] = top[n];
        if (!p.normalize && live)
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            if (key[n][i] != 0u) total[n] += expf(value_of<kType>(key[n][i]) - value_of<kType>(first[n]));
      }
      if (lane == j && live) mine[n] = top[n];
      const bool pops = key[n][0] == top[n];  // one lane's: keys are all different
#pragma unroll
      for (int i = 0; i + 1 < kEach; ++i) key[n][i] = pops ? key[n][i + 1] : key[n][i];
      key[n][kEach - 1] = pops ? Key{0u} : key[n][kEach - 1];
    }
  }
#pragma unroll
  for (int n = 0; n < kAtOnce; ++n) {
    const int at = bit + n * kWarps;
    const int expert = mine[n] != 0u ? static_cast<int>(0xFFFFu - (mine[n] & 0xFFFFu)) : -1;
    const float e = expert >= 0 ? expf(value_of<kType>(mine[n]) - value_of<kType>(first[n])) : 0.0f;
    const float sum = warp_sum(p.normalize ? e : total[n]);
    if (lane < p.k && at < tokens) {
      p.weight[(t0 + at) * p.k + lane] = expert >= 0 ? e / sum : 0.0f;
      p.expert[(t0 + at) * p.k + lane] = expert;
      if (expert >= 0) atomicOr(&mask[at / 32][expert], 1u << (at % 32));
    }
  }
}

// ------------------------------------------------------- up to eight choices: kList of them
constexpr int kList = 8;
constexpr int kLanes = 8;  // of a token

// The larger eight of two descending lists, descending (keys are all different).
template <typename T>
__device__ __forceinline__ void merge_down(T (&a)[kList], const T (&b)[kList]) {
#pragma unroll
  for (int i = 0; i < kList; ++i) a[i] = a[i] > b[kList - 1 - i] ? a[i] : b[kList - 1 - i];
#pragma unroll
  for (int d = kList / 2; d > 0; d /= 2)  // what goes up, then down, in order
#pragma unroll
    for (int i = 0; i < kList; ++i)
      if (!(i & d)) {
        const T x = a[i], y = a[i + d];
        a[i] = x > y ? x : y;
        a[i + d] = x > y ? y : x;
      }
}

// Eight neighbouring logits, the first `left` of them, as they lie in memory.
template <int kType>
struct Eight {
  static constexpr int kWords = kType == MXFP8_FP32 ? 8 : 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const RouteParams& p, int64_t t, int e, int left) {
    const int64_t at = t * p.stride + e;
    if (left >= 8 && p.wide) {
      const uint4* const from =
          kType == MXFP8_FP32
              ? reinterpret_cast<const uint4*>(static_cast<const float*>(p.logits) + at)
              : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.logits) + at);
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 u = from[i / 4];
        w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kType == MXFP8_FP32) {
        w[i] = i < left ? static_cast<const uint32_t*>(p.logits)[at + i] : 0u;
      } else {
        const uint16_t* const from = static_cast<const uint16_t*>(p.logits) + at;
        w[i] = (2 * i < left ? from[2 * i] : 0u) |
               (2 * i + 1 < left ? static_cast<uint32_t>(from[2 * i + 1]) << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ void keys(int e, int left, typename KeyOf<kType>::T (&key)[8]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kType == MXFP8_FP32) {
        key[i] = static_cast<uint64_t>(order_key(__uint_as_float(w[i]))) << 32 | (0xFFFFu - (e + i));
      } else {
        const uint32_t both = short_keys<kType>(w[i]);
        key[2 * i] = both << 16 | (0xFFFFu - (e + 2 * i));
        key[2 * i + 1] = (both & 0xFFFF0000u) | (0xFFFFu - (e + 2 * i + 1));
      }
    }
    if (left < 8)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= left) key[i] = 0u;
  }
};

// A lane's logits of the block's token `at`; none past the last token.
template <int kType, int kEights>
__device__ __forceinline__ void load_few(const RouteParams& p, int64_t t0, int tokens, int at,
                                         Eight<kType> (&eight)[kEights]) {
#pragma unroll
  for (int c = 0; c < kEights; ++c) {
    const int first = (c * kLanes + static_cast<int>(threadIdx.x) % kLanes) * 8;
    eight[c].load(p, t0 + at, first, at < tokens ? p.experts - first : 0);
  }
}
// The experts and weights of the block's token `at`, by eight lanes (past the last token
// they go along).  All of a warp.
template <int kType, int kEights>
__device__ __forceinline__ void choose_few(const RouteParams& p, int64_t t0, int tokens, int at,
                                           const Eight<kType> (&eight)[kEights],
                                           uint32_t (*mask)[MXFP8_MAX_EXPERTS]) {
  using Key = typename KeyOf<kType>::T;
  const int lane = threadIdx.x % kLanes;
  const int64_t t = t0 + at;
  const bool live = at < tokens;
  const auto first = [&](int c) { return (c * kLanes + lane) * 8; };
  const auto left = [&](int c) { return live ? p.experts - first(c) : 0; };
  Key list[kList];
  eight[0].keys(first(0), left(0), list);
  sort_down(list);
#pragma unroll
  for (int c = 1; c < kEights; ++c) {
    Key more[kList];
    eight[c].keys(first(c), left(c), more);
    sort_down(more);
    merge_down(list, more);
  }
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) {
    Key other[kList];
#pragma unroll
    for (int i = 0; i < kList; ++i) other[i] = __shfl_xor_sync(~0u, list[i], o);
    merge_down(list, other);
  }
  Key mine = list[0];  // lane j: the j-th
#pragma unroll
  for (int i = 1; i < kList; ++i) mine = lane == i ? list[i] : mine;
  const bool chosen = lane < p.k && !is_nothing<kType>(mine);
  const float top = value_of<kType>(list[0]);
  const float e = chosen ? expf(value_of<kType>(mine) - top) : 0.0f;
  float sum = e;
  if (!p.normalize) {
    sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < kEights; ++c) {
      Key key[8];
      Eight<kType> again;
      again.load(p, t, first(c), left(c));
      again.keys(first(c), left(c), key);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key[i] != 0u) sum += expf(value_of<kType>(key[i]) - top);
    }
  }
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
  if (live && lane < p.k) {
    const int expert = chosen ? static_cast<int>(0xFFFFu - (mine & 0xFFFFu)) : -1;
    p.weight[t * p.k + lane] = chosen ? e / sum : 0.0f;
    p.expert[t * p.k + lane] = expert;
    if (chosen) atomicOr(&mask[at / 32][expert], 1u << (at % 32));
  }
}

// Sum over the threads before (thread 0: 0); `sums` holds one number a warp.
__device__ __forceinline__ int before_in_block(int v, int* sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int up = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += sums[w];
  return base + inc - v;
}

// A block's tokens, for each expert as bits.
struct Masks {
  uint32_t bits[kRouteMany / 32][MXFP8_MAX_EXPERTS];
  int base[MXFP8_MAX_EXPERTS];
  int sums[kWarps];
  int routed;
};

// The slots of a block's `entries`, from the masks and, thread e, the rows of expert e (`count`:
// of all blocks, `earlier`: of those before).
__device__ __forceinline__ void place(const RouteParams& p, Masks& m, int64_t t0, int entries,
                                      int count, int earlier) {
  const int tid = threadIdx.x;
  const int begin = before_in_block(count, m.sums);
  if (tid < p.experts) {
    m.base[tid] = begin + earlier;
    if (blockIdx.x == 0) p.begin[tid] = begin;
    if (tid == p.experts - 1) {
      m.routed = begin + count;
      if (blockIdx.x == 0) p.begin[p.experts] = begin + count;
    }
  }
  __syncthreads();
  for (int i = tid; i < entries; i += kThreads) {
    const int64_t flat = t0 * p.k + i;
    const int bit = i / p.k, e = p.expert[flat];
    int slot = -1;
    if (e >= 0) {
      slot = m.base[e] + __popc(m.bits[bit / 32][e] & ((1u << (bit % 32)) - 1u));
      for (int w = 0; w < bit / 32; ++w) slot += __popc(m.bits[w][e]);
      p.row[slot] = static_cast<int32_t>(t0 + bit);
    }
    p.slot[flat] = slot;
    if (flat >= m.routed) p.row[flat] = -1;  // a slot that nothing was routed to
  }
}

// The choice; with one block the places too, else each block's counts.
template <int kType, int kEach, bool kFew>
__global__ void __launch_bounds__(kThreads)
    route_choose_kernel(const __grid_constant__ RouteParams p) {
  __shared__ Masks m;
  const int tid = threadIdx.x, warp = tid / 32, words = p.block / 32;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.block;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.block), p.tokens - t0));
  for (int w = 0; w < words; ++w) m.bits[w][tid] = 0u;
  __syncthreads();
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  if constexpr (kFew) {
    // Several times in a block of many tokens: the next logits are on their way meanwhile.
    constexpr int kEvery = kThreads / kLanes;
    constexpr bool kAhead = kEach * Eight<kType>::kWords <= 16;  // (registers)
    Eight<kType> eight[kEach];
    int at = tid / kLanes;
    load_few<kType, kEach>(p, t0, tokens, at, eight);
    for (int i = warp * (32 / kLanes); i < tokens; i += kEvery, at += kEvery) {
      Eight<kType> next[kEach];
      const bool more = i + kEvery < tokens;
      if (kAhead && more) load_few<kType, kEach>(p, t0, tokens, at + kEvery, next);
      choose_few<kType, kEach>(p, t0, tokens, at, eight, m.bits);
      if (!kAhead && more) load_few<kType, kEach>(p, t0, tokens, at + kEvery, next);
#pragma unroll
      for (int c = 0; c < kEach; ++c) eight[c] = next[c];
    }
  } else {
    // Two tokens at a time, whose logits are on their way while those before are chosen from.
    using Key = typename KeyOf<kType>::T;
    constexpr int kAtOnce = kType == MXFP8_FP32 && kEach > 8 ? 1 : 2;  // (registers)
    Key next[kAtOnce][kEach];
    const auto load = [&](int i) {
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n) {
        if (i + n * kWarps < tokens) {
          load_keys<kType, kEach>(p, t0 + i + n * kWarps, next[n]);
        } else {
#pragma unroll
          for (int q = 0; q < kEach; ++q) next[n][q] = 0u;
        }
      }
    };
    load(warp);
    for (int i = warp; i < tokens; i += kAtOnce * kWarps) {
      Key key[kAtOnce][kEach];
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n)
#pragma unroll
        for (int q = 0; q < kEach; ++q) key[n][q] = next[n][q];
      load(i + kAtOnce * kWarps);
      choose<kType, kEach, kAtOnce>(p, t0, tokens, i, key, m.bits);
    }
  }
  __syncthreads();
  int count = 0;
  for (int w = 0; w < words; ++w) count += __popc(m.bits[w][tid]);
  if (gridDim.x > 1) {
    if (tid < p.experts) p.counts[static_cast<size_t>(blockIdx.x) * p.experts + tid] = count;
    return;
  }
  place(p, m, t0, max(tokens, 0) * p.k, count, 0);
}

// The places: kSums from the sums of the counts before each block, else from the counts.
template <bool kSums>
__global__ void __launch_bounds__(kThreads)
    route_place_kernel(const __grid_constant__ RouteParams p) {
  __shared__ Masks m;
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.block;
  const int entries =
      static_cast<int>(min(static_cast<int64_t>(p.block), p.tokens - t0)) * p.k;
  for (int w = 0; w < p.block / 32; ++w) m.bits[w][tid] = 0u;
  __syncthreads();
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  int count = 0, earlier = 0;
  if (tid < p.experts) {
    if constexpr (kSums) {
      count = p.counts[static_cast<size_t>(gridDim.x) * p.experts + tid];
      earlier = p.counts[static_cast<size_t>(blockIdx.x) * p.experts + tid];
    } else {
      const int blocks = gridDim.x, mine = blockIdx.x;
      for (int b = 0; b < blocks; b += 16) {  // all under way together
        int c[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = b + i < blocks ? p.counts[(b + i) * p.experts + tid] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          count += c[i];
          if (b + i < mine) earlier += c[i];
        }
      }
    }
  }
  for (int i = tid; i < entries; i += kThreads) {
    const int e = p.expert[t0 * p.k + i];
    if (e >= 0) atomicOr(&m.bits[i / p.k / 32][e], 1u << (i / p.k % 32));
  }
  __syncthreads();
  place(p, m, t0, entries, count, earlier);
}

// Each expert's counts become those of the blocks before, in place, and the row after
// the last block's the sum.  A block of 32 x 32: 32 experts, whose blocks the 32 rows of
// threads take in turn.
__global__ void __launch_bounds__(1024) route_sum_kernel(int32_t* counts, int experts, int blocks) {
  __shared__ int sums[32][33];
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x % 32, part = threadIdx.x / 32, e = blockIdx.x * 32 + lane;
  const int each = (blocks + 31) / 32, from = min(part * each, blocks), to = min(from + each, blocks);
  const auto load = [&](int b, int (&c)[8]) {  // eight at a time, all under way together
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = e < experts && b + i < to ? counts[static_cast<size_t>(b + i) * experts + e] : 0;
  };
  int c[8], sum = 0;
  for (int b = from; b < to; b += 8) {
    load(b, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += c[i];
  }
  sums[part][lane] = sum;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int q = 0; q < 31; ++q)
    if (q < part) before += sums[q][lane];
  if (e >= experts) return;
  for (int b = from; b < to; b += 8) {
    if (each > 8) load(b, c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (b + i < to) {
        counts[static_cast<size_t>(b + i) * experts + e] = before;
        before += c[i];
      }
  }
  if (part == 31) counts[static_cast<size_t>(blocks) * experts + e] = before;
}

constexpr int kCombineThreads = 256;

template <int kAtOnce>
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const __grid_constant__ CombineParams p) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const uint32_t i = blockIdx.x * static_cast<uint32_t>(kCombineThreads) + threadIdx.x;
  if (i >= p.items) return;
  const uint32_t per_row = static_cast<uint32_t>(p.n) / 8;
  const uint32_t t = i / per_row, c = (i - t * per_row) * 8;
  const int32_t* slots = p.slot + static_cast<size_t>(t) * p.k;
  const float* weights = p.weight + static_cast<size_t>(t) * p.k;
  float acc[8] = {};
  if (p.add) {
    const uint4 u = *reinterpret_cast<const uint4*>(p.add + static_cast<size_t>(t) * p.n + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[2 * q] = __uint_as_float(w[q] << 16);
      acc[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
  for (int j0 = 0; j0 < p.k; j0 += kAtOnce) {
    uint4 u[kAtOnce];
    float g[kAtOnce];
    bool live[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int s = j0 + j < p.k ? slots[j0 + j] : -1;
      live[j] = s >= 0 && s < p.slots;
      if (!live[j] && s != -1 && p.flags) atomicOr(p.flags, MXFP8_FLAG_BAD_INDEX);
      g[j] = 0.0f;
      u[j] = make_uint4(0u, 0u, 0u, 0u);
      if (live[j]) {
        g[j] = weights[j0 + j];
        u[j] = ptx::ld_once_v4(p.y + static_cast<int64_t>(s) * p.y_stride + c);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (!live[j]) continue;
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[2 * q] = fmaf(g[j], __uint_as_float(w[q] << 16), acc[2 * q]);
        acc[2 * q + 1] = fmaf(g[j], __uint_as_float(w[q] & 0xFFFF0000u), acc[2 * q + 1]);
      }
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * q], acc[2 * q + 1]);
    w[q] = *reinterpret_cast<const uint32_t*>(&b);
  }
  ptx::st_v4(p.out + static_cast<size_t>(t) * p.n + c, make_uint4(w[0], w[1], w[2], w[3]));
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), uint32_t blocks, int threads, cudaStream_t stream,
                   Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(threads);
  cfg.gridDim = dim3(blocks);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// kEach: keys a lane has, or where there are few choices eights of them.
template <int kType, int kEach, bool kFew>
cudaError_t route_as(const RouteParams& p, cudaStream_t stream) {
  const uint32_t blocks =
      static_cast<uint32_t>(p.tokens <= p.block ? 1 : (p.tokens + p.block - 1) / p.block);
  cudaError_t e = launch(route_choose_kernel<kType, kEach, kFew>, blocks, kThreads, stream, p);
  if (e != cudaSuccess || blocks == 1) return e;
  if (blocks <= 64) return launch(route_place_kernel<false>, blocks, kThreads, stream, p);
  e = launch(route_sum_kernel, static_cast<uint32_t>((p.experts + 31) / 32), 1024, stream, p.counts,
             p.experts, static_cast<int>(blocks));
  if (e != cudaSuccess) return e;
  return launch(route_place_kernel<true>, blocks, kThreads, stream, p);
}
template <int kType>
cudaError_t route_for(const RouteParams& p, cudaStream_t stream) {
  if (p.k <= kList) {
    if (p.experts <= 64) return route_as<kType, 1, true>(p, stream);
    if (p.experts <= 128) return route_as<kType, 2, true>(p, stream);
    if (p.experts <= 256) return route_as<kType, 4, true>(p, stream);
    return route_as<kType, 8, true>(p, stream);
  }
  return p.experts <= 256 ? route_as<kType, 8, false>(p, stream)
                          : route_as<kType, 16, false>(p, stream);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  switch (p.type) {
    case MXFP8_BF16: return route_for<MXFP8_BF16>(p, stream);
    case MXFP8_FP16: return route_for<MXFP8_FP16>(p, stream);
    default: return route_for<MXFP8_FP32>(p, stream);
  }
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream) {
  const uint32_t blocks = (p.items + kCombineThreads - 1) / kCombineThreads;
  return p.k <= 4 ? launch(combine_kernel<4>, blocks, kCombineThreads, stream, p)
                  : launch(combine_kernel<8>, blocks, kCombineThreads, stream, p);
}

}  // namespace mxfp8
