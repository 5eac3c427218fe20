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
// rows that see it NaN.  Statistics and sums are FP32.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kRope = 64;

__device__ __forceinline__ float bf16(uint16_t bits) {
  return __uint_as_float(static_cast<uint32_t>(bits) << 16);
}

__device__ __forceinline__ void raise(int32_t* flags) {
  if (flags != nullptr)
    atomicOr(reinterpret_cast<unsigned int*>(flags), MXFP8_FLAG_BAD_INDEX);
}

// One CTA per (row, head): each warp takes every eighth token, lane = every
// 32nd element.
template <int kLatent>
__global__ void __launch_bounds__(256) attend_rows_kernel(const __grid_constant__ LatentParams p) {
  constexpr int kWidth = kLatent + kRope;
  constexpr int kPer = kWidth / 32;
  __shared__ float stats[8][2];
  __shared__ float sums[8][kLatent];
  ptx::grid_dependency_wait();
  const int row = blockIdx.x / p.heads;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const size_t qrow = blockIdx.x;
  int b = -1;
  for (int i = 0; i < p.requests; ++i)
    if (p.row_begin[i] <= row && row < p.row_begin[i + 1]) b = i;
  float q[kPer], acc[kPer - 2] = {};
  for (int i = 0; i < kPer; ++i) q[i] = bf16(p.q[qrow * kWidth + i * 32 + lane]);
  float top = -INFINITY, total = 0.0f;
  if (b >= 0) {
    const int t = row - p.row_begin[b];
    const int drafts = min(p.row_begin[b + 1], p.rows) - p.row_begin[b];
    if (p.row_begin[b] < 0 || p.row_begin[b + 1] > p.rows) raise(p.flags);
    const int length = min(max(p.lengths[b], 0), p.table_width * p.page_size);
    if (length != p.lengths[b]) raise(p.flags);
    const int context = max(length - drafts, 0);
    const uint64_t tree = p.tree != nullptr ? static_cast<uint64_t>(p.tree[row]) : 0;
    for (int at = warp; at < length; at += 8) {
      const int d = at - context;
      if (d >= 0 && !(p.tree != nullptr ? d < 64 && (tree >> d & 1) : d <= t)) continue;
      const int page = p.table[static_cast<size_t>(b) * p.table_width + at / p.page_size];
      const bool known = page >= 0 && page < p.pages;
      if (!known) raise(p.flags);
      const uint16_t* c = p.cache + (known ? page : 0) * p.page_stride +
                          at % p.page_size * p.token_stride;
      float kv[kPer], z = 0.0f;
      for (int i = 0; i < kPer; ++i) {
        kv[i] = known ? bf16(c[i * 32 + lane]) : 0.0f;
        z = fmaf(q[i], kv[i], z);
      }
      for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(~0u, z, o);
      z *= p.scale_log2;
      bool finite = true;
      for (int i = 0; i < kPer - 2; ++i) finite = finite && isfinite(kv[i]);
      if (d >= 0 && !__all_sync(~0u, finite)) z = NAN;
      const float next = fmaxf(top, z);
      const float keep = top == next ? 1.0f : exp2f(top - next);
      const float e = exp2f(z - next);
      total = total * keep + e;
      for (int i = 0; i < kPer - 2; ++i) acc[i] = acc[i] * keep + e * kv[i];
      top = next;
    }
  }
  if (lane == 0) {
    stats[warp][0] = top;
    stats[warp][1] = total;
  }
  for (int i = 0; i < kPer - 2; ++i) sums[warp][i * 32 + lane] = acc[i];
  __syncthreads();
  float best = -INFINITY;
  for (int i = 0; i < 8; ++i) best = fmaxf(best, stats[i][0]);
  for (int c = threadIdx.x; c < kLatent; c += 256) {
    float sum = 0.0f, all = 0.0f;
    for (int i = 0; i < 8; ++i) {
      if (stats[i][1] == 0.0f) continue;
      const float f = exp2f(stats[i][0] - best);
      sum += f * sums[i][c];
      all += f * stats[i][1];
    }
    p.out[qrow * kLatent + c] =
        __bfloat16_as_ushort(__float2bfloat16_rn(all == 0.0f ? 0.0f : sum / all));
  }
}

}  // namespace

cudaError_t launch_latent_attend(const LatentParams& p, int latent, cudaStream_t stream) {
  const int grid = p.rows * p.heads;
  if (latent == 512)
    attend_rows_kernel<512><<<grid, 256, 0, stream>>>(p);
  else
    attend_rows_kernel<256><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mxfp8
