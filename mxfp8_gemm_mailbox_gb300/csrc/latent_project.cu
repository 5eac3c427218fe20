// The products that lead into and out of the latent space, one matrix a head:
//
//   query:  q[t][h][c] = sum_d W[h][c][d] q_nope[t][h][d], the rotary part
//           copied behind it (BF16);
//   values: y[t][h][v] = sum_c W[h][v][c] o[t][h][c], rounded to MXFP8 along
//           the row [h][v] in blocks of 32, which is the projection's x.
//
// Sums in FP32.  A block's scale is the smallest power of two under which no
// element passes 448, E4M3's largest, so none saturates; the elements are
// rounded to nearest, ties to even.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kRope = 64;

__device__ __forceinline__ float bf16(uint16_t bits) {
  return __uint_as_float(static_cast<uint32_t>(bits) << 16);
}

// The E8M0 code of a block whose largest magnitude is `top`: 127 for a block
// of zeros; top = f 2^E (1 <= f < 2) takes E - 8 for f <= 1.75, else E - 7.
__device__ __forceinline__ uint32_t scale_code(float top) {
  const uint32_t bits = __float_as_uint(top);
  if (bits == 0u) return 127u;
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, 0), 254));
}

__device__ __forceinline__ uint8_t to_e4m3(float v, uint32_t code) {
  // v 2^(127 - code) in two exact halves (one power may be past FP32's range).
  const int e = 127 - static_cast<int>(code);
  const float s = __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
  const float r = __uint_as_float(static_cast<uint32_t>(127 + e - e / 2) << 23);
  return __nv_cvt_float_to_fp8(v * s * r, __NV_SATFINITE, __NV_E4M3);
}

// One warp per 32 outputs of one head and row; lane = output.
template <bool kQuery>
__global__ void head_products_kernel(const uint16_t* __restrict__ in,
                                     const uint16_t* __restrict__ rope,
                                     const uint16_t* __restrict__ w, uint16_t* __restrict__ q,
                                     uint8_t* __restrict__ x, uint8_t* __restrict__ x_scale,
                                     int heads, int inner, int outer) {
  ptx::grid_dependency_wait();
  const int t = blockIdx.z, h = blockIdx.y, lane = threadIdx.x;
  const int j = blockIdx.x * 32 + lane;
  const size_t th = static_cast<size_t>(t) * heads + h;
  if (kQuery && j >= outer) {
    const int d = j - outer;
    q[th * (outer + kRope) + j] = rope[th * kRope + d];
    return;
  }
  const uint16_t* row = w + (static_cast<size_t>(h) * outer + j) * inner;
  float sum = 0.0f;
  for (int i = 0; i < inner; ++i) sum = fmaf(bf16(row[i]), bf16(in[th * inner + i]), sum);
  if (kQuery) {
    q[th * (outer + kRope) + j] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
  } else {
    float top = fabsf(sum);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const uint32_t code = scale_code(top);
    x[th * outer + j] = to_e4m3(sum, code);
    if (lane == 0) x_scale[th * (outer / 32) + blockIdx.x] = static_cast<uint8_t>(code);
  }
}

}  // namespace

cudaError_t launch_latent_query(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w,
                                uint16_t* q, int rows, int heads, int nope, int latent,
                                cudaStream_t stream) {
  head_products_kernel<true><<<dim3((latent + kRope) / 32, heads, rows), 32, 0, stream>>>(
      q_nope, q_rope, w, q, nullptr, nullptr, heads, nope, latent);
  return cudaGetLastError();
}

cudaError_t launch_latent_values(const uint16_t* o, const uint16_t* w, uint8_t* x,
                                 uint8_t* x_scale, int rows, int heads, int latent, int value,
                                 cudaStream_t stream) {
  head_products_kernel<false><<<dim3(value / 32, heads, rows), 32, 0, stream>>>(
      o, nullptr, w, nullptr, x, x_scale, heads, latent, value);
  return cudaGetLastError();
}

}  // namespace mxfp8
