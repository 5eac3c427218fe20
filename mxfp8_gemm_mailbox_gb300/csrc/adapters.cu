// Low-rank adapters of the rows of one projection call:
//
//   delta[t][n] = gain[i] sum_j B[i][n][j] (sum_k A[i][j][k] x[t][k]),
//   i = which[t], j < ranks[i]
//
// with x the MXFP8 row that the projection itself reads (E4M3 elements, one
// E8M0 scale per 32), A and B BF16 and both sums in FP32.  The publishing
// GEMM adds delta to its compensated sum before the one rounding of C, so C is
// what a weight with the adapter merged into it would give.
//
// Both products read their matrix once for one row of activations each: bound
// by HBM (8 rows with adapters of their own, rank 64, N = 7168, K = 16384: 16.8
// MB of A, 7.3 MB of B beside the projection's 121 MB).  The first, three blocks
// an SM, has all of A on its way at once and takes 5.3 us of that call.  The
// second, one block an SM of 4 warps x 72 registers a thread and next to no
// shared memory, leaves room for two of the GEMM's blocks and runs under the
// GEMM's weight stream: both let their dependents launch at once, and the GEMM
// waits for delta in its epilogue alone.  30.6 us a call (21.2 without adapters;
// 145 MB are 21.2 us at the copy rate): the GEMM's blocks come when the first
// kernel's leave.  35 with two or three blocks of the second an SM (they come
// after the first kernel, and the GEMM's after them), 30.9 with smaller blocks of
// the first that the GEMM's fit beside.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "even_share.h"
#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

__device__ __forceinline__ float e8m0(uint32_t code) {
  if (code == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(code == 0u ? 0x00400000u : code << 23);
}

// The adapter of row t, or -1; an index outside -1..count-1 raises the flag
// and counts as none.
__device__ __forceinline__ int adapter_of(const AdapterParams& p, int t) {
  const int i = p.which[t];
  if (i >= -1 && i < p.count) return i;
  atomicOr(reinterpret_cast<unsigned int*>(p.flags), MXFP8_FLAG_BAD_INDEX);
  return -1;
}

__device__ __forceinline__ int rank_of(const AdapterParams& p, int i) {
  return p.ranks == nullptr ? p.rank : min(max(p.ranks[i], 0), p.rank);
}

constexpr int kSteps = 3;          // loads of a row of A a lane has on its way
constexpr int kPiece = kSteps * 256;  // numbers of a row of x a warp multiplies
constexpr int kRowsOfA = 4;        // rows of A a warp takes
constexpr int kInnerThreads = 256;

__host__ __device__ constexpr int pieces_of(int k) { return (k + kPiece - 1) / kPiece; }

__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) {
  return __uint_as_float(w & 0xFFFF0000u);
}

// inner[t][piece][j]: lane l of a warp takes numbers 8 l .. 8 l + 7 of every 256
// of its piece of K, for four rows of A; a warp's items are (row t, piece, four
// rows), every gridDim.x x 8 warps.
__device__ __forceinline__ void inner_item(const AdapterParams& p, int t, int piece, int j0,
                                           int lane) {
  const int i = adapter_of(p, t);
  if (i < 0) return;
  const int rank = rank_of(p, i);
  if (j0 >= rank) return;
  const int k0 = piece * kPiece + lane * 8;
  uint4 a[kRowsOfA][kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int r = 0; r < kRowsOfA; ++r) {
      a[r][s] = make_uint4(0u, 0u, 0u, 0u);
      if (j0 + r < rank && k0 + s * 256 < p.k)
        a[r][s] = ptx::ld_once_v4(p.a + (static_cast<size_t>(i) * p.rank + j0 + r) * p.k + k0 + s * 256);
    }
  float sum[kRowsOfA] = {};
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int k = k0 + s * 256;
    if (k >= p.k) continue;
    const uint2 codes = *reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(t) * p.k + k);
    const float scale = e8m0(p.x_scale[static_cast<size_t>(t) * (p.k / 32) + k / 32]);
    __nv_fp8x4_e4m3 quad[2];
    quad[0].__x = codes.x;
    quad[1].__x = codes.y;
    const float4 lo = static_cast<float4>(quad[0]), hi = static_cast<float4>(quad[1]);
    const float x[8] = {lo.x * scale, lo.y * scale, lo.z * scale, lo.w * scale,
                        hi.x * scale, hi.y * scale, hi.z * scale, hi.w * scale};
#pragma unroll
    for (int r = 0; r < kRowsOfA; ++r) {
      const uint32_t w[4] = {a[r][s].x, a[r][s].y, a[r][s].z, a[r][s].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sum[r] = fmaf(low_bf16(w[q]), x[2 * q], sum[r]);
        sum[r] = fmaf(high_bf16(w[q]), x[2 * q + 1], sum[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsOfA; ++r)
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[r] += __shfl_xor_sync(~0u, sum[r], o);
  if (lane < kRowsOfA && j0 + lane < rank) {
    const float v = lane == 0 ? sum[0] : lane == 1 ? sum[1] : lane == 2 ? sum[2] : sum[3];
    p.inner[(static_cast<size_t>(t) * pieces_of(p.k) + piece) * p.rank + j0 + lane] = v;
  }
}

__global__ void __launch_bounds__(kInnerThreads, 3)
    adapter_inner_kernel(const __grid_constant__ AdapterParams p) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();  // past the wait: the next kernels may read the call's inputs at once
  const int groups = (p.rank + kRowsOfA - 1) / kRowsOfA, pieces = pieces_of(p.k);
  const int items = p.m * pieces * groups, warps = gridDim.x * (kInnerThreads / 32);
  for (int at = blockIdx.x * (kInnerThreads / 32) + threadIdx.x / 32; at < items; at += warps)
    inner_item(p, at / (pieces * groups), at / groups % pieces, at % groups * kRowsOfA,
               threadIdx.x % 32);
}

constexpr int kDeltaThreads = 128;
constexpr int kDeltaLoads = 8;  // of a thread, at once

// delta[t][n]: kLanes lanes share a row of B, 16 bytes (8 numbers) each a turn.
// A block's items are (row t, kDeltaLoads x 128 / kLanes outputs), in a row: it
// gathers the products with A once, for mostly one t.  (Beside the GEMM's weight
// stream such a round trip takes 2 to 3 us; with every gridDim.x-th item this
// kernel outlasted the GEMM by 1 us at 8 rows of rank 64.)
template <int kLanes>
__global__ void __launch_bounds__(kDeltaThreads, 7)
    adapter_delta_kernel(const __grid_constant__ AdapterParams p) {
  __shared__ float inner[MXFP8_MAX_ADAPTER_RANK];
  ptx::launch_dependents();
  constexpr int kAtOnce = kDeltaThreads / kLanes;  // outputs a turn
  constexpr int kOutputs = kAtOnce * kDeltaLoads;
  const int tid = threadIdx.x, sub = tid % kLanes;
  const int blocks = (p.n + kOutputs - 1) / kOutputs, items = p.m * blocks;
  const int rank8 = (p.rank + 7) & ~7, pieces = pieces_of(p.k);
  int have = -1;  // the row whose products with A are in `inner`
  const EvenShare share = even_share(items, blockIdx.x, gridDim.x);
  for (int item = share.first; item < share.last; ++item) {
    const int t = item / blocks, n0 = item % blocks * kOutputs + tid / kLanes;
    const int i = adapter_of(p, t);
    const int rank = i < 0 ? 0 : rank_of(p, i);
    const uint16_t* b = p.b + (static_cast<size_t>(max(i, 0)) * p.n + n0) * rank8 + sub * 8;
    // The first turn's part of B, before the wait for the products with A.
    uint4 w[kDeltaLoads];
    const bool live = sub * 8 < rank;
#pragma unroll
    for (int l = 0; l < kDeltaLoads; ++l)
      if (live && n0 + l * kAtOnce < p.n)
        w[l] = ptx::ld_once_v4(b + static_cast<size_t>(l) * kAtOnce * rank8);
    if (have < 0) ptx::grid_dependency_wait();
    if (have != t) {
      if (have >= 0) __syncthreads();
      for (int j = tid; j < rank; j += kDeltaThreads) {
        float sum = 0.0f;
#pragma unroll 8
        for (int piece = 0; piece < pieces; ++piece)
          sum += p.inner[(static_cast<size_t>(t) * pieces + piece) * p.rank + j];
        inner[j] = sum;
      }
      __syncthreads();
      have = t;
    }
    const float gain = i < 0 || p.gain == nullptr ? 1.0f : p.gain[i];
    float sum[kDeltaLoads] = {};
    for (int j0 = sub * 8; j0 < rank; j0 += kLanes * 8) {
      if (j0 != sub * 8) {
#pragma unroll
        for (int l = 0; l < kDeltaLoads; ++l)
          if (n0 + l * kAtOnce < p.n)
            w[l] = ptx::ld_once_v4(b + static_cast<size_t>(l) * kAtOnce * rank8 + j0 - sub * 8);
      }
      // (Columns past the adapter's rank may hold anything.)
      const int left = rank - j0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v0 = inner[min(j0 + 2 * q, rank - 1)];
        const float v1 = inner[min(j0 + 2 * q + 1, rank - 1)];
#pragma unroll
        for (int l = 0; l < kDeltaLoads; ++l) {
          const uint32_t c = q == 0 ? w[l].x : q == 1 ? w[l].y : q == 2 ? w[l].z : w[l].w;
          if (2 * q < left) sum[l] = fmaf(low_bf16(c), v0, sum[l]);
          if (2 * q + 1 < left) sum[l] = fmaf(high_bf16(c), v1, sum[l]);
        }
      }
    }
#pragma unroll
    for (int l = 0; l < kDeltaLoads; ++l) {
#pragma unroll
      for (int o = kLanes / 2; o; o /= 2) sum[l] += __shfl_xor_sync(~0u, sum[l], o);
      const int n = n0 + l * kAtOnce;
      if (sub == 0 && n < p.n) p.delta[static_cast<size_t>(t) * p.n + n] = sum[l] * gain;
    }
  }
  if (have < 0) ptx::grid_dependency_wait();
}

// An SM's split between cache and shared memory changes only while it is idle,
// so both kernels ask for the GEMM's: its blocks could not join them otherwise.
template <auto* kKernel>
cudaError_t share_sm(int device) {
  static std::mutex mutex;
  static bool done[64] = {};
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mutex);
  if (done[device]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      kKernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  done[device] = e == cudaSuccess;
  return e;
}

template <int kLanes>
cudaError_t launch_delta(const AdapterParams& p, cudaLaunchConfig_t cfg, int device, int sms) {
  constexpr int kOutputs = kDeltaThreads / kLanes * kDeltaLoads;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(p.m * ((p.n + kOutputs - 1) / kOutputs), sms)));
  cfg.blockDim = dim3(kDeltaThreads);
  const cudaError_t e = share_sm<&adapter_delta_kernel<kLanes>>(device);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, adapter_delta_kernel<kLanes>, p);
}

}  // namespace

size_t adapter_inner_floats(int k, int rank) {
  return (static_cast<size_t>(kRows) * pieces_of(k) * rank + 3) & ~size_t{3};
}

cudaError_t launch_adapters(const AdapterParams& p, int device, int sms, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int items = p.m * pieces_of(p.k) * ((p.rank + kRowsOfA - 1) / kRowsOfA);
  constexpr int kWarps = kInnerThreads / 32;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min((items + kWarps - 1) / kWarps, 3 * sms)));
  cfg.blockDim = dim3(kInnerThreads);
  cudaError_t e = share_sm<&adapter_inner_kernel>(device);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, adapter_inner_kernel, p);
  if (e != cudaSuccess) return e;
  // Lanes to a row of B: what its 16-byte pieces fill, at most 8 (rank 64).
  if (p.rank <= 8) return launch_delta<1>(p, cfg, device, sms);
  if (p.rank <= 16) return launch_delta<2>(p, cfg, device, sms);
  if (p.rank <= 32) return launch_delta<4>(p, cfg, device, sms);
  return launch_delta<8>(p, cfg, device, sms);
}

}  // namespace mxfp8
