// Low-rank adapters of the rows of one projection call:
//
//   delta[t][n] = gain[i] sum_j B[i][n][j] (sum_k A[i][j][k] x[t][k]),
//   i = which[t], j < ranks[i]
//
// with x the MXFP8 row that the projection itself reads (E4M3 elements, one
// E8M0 scale per 32), A and B BF16 and both sums in FP32.  The publishing
// GEMM adds delta to its compensated sum before the one rounding of C, so C is
// what a weight with the adapter merged into it would give.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

__device__ __forceinline__ float e8m0(uint32_t code) {
  if (code == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(code == 0u ? 0x00400000u : code << 23);
}

__device__ __forceinline__ float e4m3(uint8_t code) {
  __nv_fp8_e4m3 v;
  v.__x = code;
  return static_cast<float>(v);
}

__device__ __forceinline__ float bf16(uint16_t bits) {
  return __uint_as_float(static_cast<uint32_t>(bits) << 16);
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

// One warp per (row, j).
__global__ void adapter_inner_kernel(const __grid_constant__ AdapterParams p) {
  ptx::grid_dependency_wait();
  const int t = blockIdx.y;
  const int j = blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int i = adapter_of(p, t);
  if (i < 0 || j >= rank_of(p, i)) return;
  const uint16_t* a = p.a + (static_cast<size_t>(i) * p.rank + j) * p.k;
  const uint8_t* x = p.x + static_cast<size_t>(t) * p.k;
  const uint8_t* xs = p.x_scale + static_cast<size_t>(t) * (p.k / 32);
  float sum = 0.0f;
  for (int k = lane; k < p.k; k += 32) sum = fmaf(bf16(a[k]), e4m3(x[k]) * e8m0(xs[k / 32]), sum);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) p.inner[t * p.rank + j] = sum;
}

// One thread per (row, n).
__global__ void adapter_delta_kernel(const __grid_constant__ AdapterParams p) {
  ptx::grid_dependency_wait();
  const int t = blockIdx.y;
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= p.n) return;
  const int i = adapter_of(p, t);
  float sum = 0.0f;
  if (i >= 0) {
    const int rank = rank_of(p, i);
    const int rank8 = (p.rank + 7) & ~7;
    const uint16_t* b = p.b + (static_cast<size_t>(i) * p.n + n) * rank8;
    for (int j = 0; j < rank; ++j) sum = fmaf(bf16(b[j]), p.inner[t * p.rank + j], sum);
    if (p.gain != nullptr) sum *= p.gain[i];
  }
  p.delta[static_cast<size_t>(t) * p.n + n] = sum;
}

}  // namespace

size_t adapter_inner_floats(int, int rank) { return static_cast<size_t>(kRows) * ((rank + 3) & ~3); }

cudaError_t launch_adapters(const AdapterParams& p, cudaStream_t stream) {
  adapter_inner_kernel<<<dim3((p.rank + 7) / 8, p.m), 256, 0, stream>>>(p);
  adapter_delta_kernel<<<dim3((p.n + 255) / 256, p.m), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mxfp8
