// Around the experts' products: the choice of each token's experts, the tokens
// in the experts' order, and the sum of what the experts gave.
//
// Route.  Token t's experts are those of its k largest logits, ties to the
// lowest index; its weights exp(z_e - z_max) over the sum of those (or of all).
// A slot is a row of the experts' products: slots are numbered by expert, then
// by token.  A logit of -infinity is not chosen: such an entry has no slot.
//
// A warp takes a token, its logits in registers.  A value's order is that of an
// integer made of its bits, so a step of the choice is two warp reductions: the
// largest key, and the lowest index that has it.  An expert appears once at
// most among a token's, so a block of 128 tokens is, for each expert, a mask of
// 128 bits: its population is the block's count, and that of the bits below a
// token the token's place.  Nothing depends on the order of atomics.  One block
// does all of up to 128 tokens; for more a second kernel adds the counts of the
// blocks before.
//
// Combine.  out[t] = add[t] + sum_j weight[t][j] y[slot[t][j]], in FP32, j
// ascending, rounded once; a thread has 8 numbers of a row, and its loads are
// all under way at once.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kTokens = kRouteTokens;  // of a block
constexpr int kMaskWords = kTokens / 32;
static_assert(kThreads >= MXFP8_MAX_EXPERTS, "a thread an expert");

// Larger values have larger keys; +0 and -0 one; NaN the largest of all.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return ~0u;
  return (b >> 31) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kNothing = 0x007FFFFFu;  // order_key(-infinity)

__device__ __forceinline__ float logit(const RouteParams& p, int64_t t, int e) {
  const int64_t at = t * p.stride + e;
  if (p.type == MXFP8_FP32) return static_cast<const float*>(p.logits)[at];
  const uint16_t h = static_cast<const uint16_t*>(p.logits)[at];
  if (p.type == MXFP8_BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Token t's experts and weights; the chosen experts' bits in `mask`.
template <int kEach>
__device__ void choose(const RouteParams& p, int64_t t, int bit, uint32_t (*mask)[MXFP8_MAX_EXPERTS]) {
  const int lane = threadIdx.x % 32;
  float z[kEach];
  uint32_t key[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = lane + 32 * i;
    z[i] = e < p.experts ? logit(p, t, e) : -INFINITY;
    key[i] = e < p.experts ? order_key(z[i]) : 0u;
  }
  float first = 0.0f, mine = 0.0f;  // lane j: the j-th chosen logit
  int expert = -1;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < kEach; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(~0u, best);
    if (top <= kNothing) break;  // -infinity from here on
    uint32_t at = ~0u;
#pragma unroll
    for (int i = kEach - 1; i >= 0; --i)
      if (key[i] == top) at = lane + 32 * i;
    at = __reduce_min_sync(~0u, at);
    float value = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (lane + 32 * i == at) {
        value = z[i];
        key[i] = 0u;
      }
    value = __shfl_sync(~0u, value, at % 32);
    if (j == 0) first = value;
    if (lane == j) {
      mine = value;
      expert = static_cast<int>(at);
    }
  }
  float e = expert >= 0 ? expf(mine - first) : 0.0f;
  float total = e;
  if (!p.normalize) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (lane + 32 * i < p.experts) total += expf(z[i] - first);
  }
  total = warp_sum(total);
  if (lane < p.k) {
    p.weight[t * p.k + lane] = expert >= 0 ? e / total : 0.0f;
    p.expert[t * p.k + lane] = expert;
    if (expert >= 0) atomicOr(&mask[bit / 32][expert], 1u << (bit % 32));
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

// kStep 0: all of a call with one block.  1: the choice, and each block's
// counts.  2: the places.
template <int kStep, int kEach>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ uint32_t mask[kMaskWords][MXFP8_MAX_EXPERTS];
  __shared__ int base[MXFP8_MAX_EXPERTS];
  __shared__ int sums[kWarps];
  __shared__ int routed;
  const int tid = threadIdx.x, warp = tid / 32;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(kTokens), p.tokens - t0));
  const int entries = max(tokens, 0) * p.k;
  for (int i = tid; i < kMaskWords * MXFP8_MAX_EXPERTS; i += kThreads) (&mask[0][0])[i] = 0u;
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  __syncthreads();
  if constexpr (kStep != 2) {
    for (int i = warp; i < tokens; i += kWarps) choose<kEach>(p, t0 + i, i, mask);
  } else {
    for (int i = tid; i < entries; i += kThreads) {
      const int e = p.expert[t0 * p.k + i];
      if (e >= 0) atomicOr(&mask[i / p.k / 32][e], 1u << (i / p.k % 32));
    }
  }
  __syncthreads();
  int count = 0;
  if (tid < p.experts)
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) count += __popc(mask[w][tid]);
  if constexpr (kStep == 1) {
    if (tid < p.experts) p.counts[static_cast<size_t>(blockIdx.x) * p.experts + tid] = count;
    return;
  }
  int all = count, earlier = 0;
  if constexpr (kStep == 2) {
    all = 0;
    const int blocks = gridDim.x, mine = blockIdx.x;
    if (tid < p.experts)
#pragma unroll 8
      for (int b = 0; b < blocks; ++b) {
        const int c = p.counts[static_cast<size_t>(b) * p.experts + tid];
        all += c;
        if (b < mine) earlier += c;
      }
  }
  const int begin = before_in_block(all, sums);
  if (tid < p.experts) {
    base[tid] = begin + earlier;
    if (blockIdx.x == 0) p.begin[tid] = begin;
    if (tid == p.experts - 1) {
      routed = begin + all;
      if (blockIdx.x == 0) p.begin[p.experts] = begin + all;
    }
  }
  __syncthreads();
  for (int i = tid; i < entries; i += kThreads) {
    const int64_t flat = t0 * p.k + i;
    const int bit = i / p.k, e = p.expert[flat];
    int slot = -1;
    if (e >= 0) {
      slot = base[e] + __popc(mask[bit / 32][e] & ((1u << (bit % 32)) - 1u));
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w)
        if (w < bit / 32) slot += __popc(mask[w][e]);
      p.row[slot] = static_cast<int32_t>(t0 + bit);
    }
    p.slot[flat] = slot;
    if (flat >= routed) p.row[flat] = -1;  // a slot that nothing was routed to
  }
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

template <typename Params>
cudaError_t launch(void (*kernel)(Params), uint32_t blocks, int threads, const Params& p,
                   cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(threads);
  cfg.gridDim = dim3(blocks);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int kEach>
cudaError_t route_as(const RouteParams& p, cudaStream_t stream) {
  const uint32_t blocks = static_cast<uint32_t>((p.tokens + kTokens - 1) / kTokens);
  if (blocks <= 1) return launch(route_kernel<0, kEach>, 1, kThreads, p, stream);
  const cudaError_t e = launch(route_kernel<1, kEach>, blocks, kThreads, p, stream);
  if (e != cudaSuccess) return e;
  return launch(route_kernel<2, 1>, blocks, kThreads, p, stream);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  if (p.experts <= 64) return route_as<2>(p, stream);
  if (p.experts <= 256) return route_as<8>(p, stream);
  return route_as<16>(p, stream);
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream) {
  const uint32_t blocks = (p.items + kCombineThreads - 1) / kCombineThreads;
  return p.k <= 4 ? launch(combine_kernel<4>, blocks, kCombineThreads, p, stream)
                  : launch(combine_kernel<8>, blocks, kCombineThreads, p, stream);
}

}  // namespace mxfp8
