// Rows into MXFP8 or MXFP4 and back:
//
//   block b of row r:  s = the smallest power of two with max |x| / s <= top,
//                      codes = round(x / s)   (top 448: E4M3, 6: E2M1)
//
// x BF16, FP16 or FP32; the row that output row r is made of may be named by an
// index (the rows of a token's experts).  An element that is not finite is NaN
// in E4M3 and no part of its block's scale; E2M1 has no NaN, so there the block
// takes the scale NaN (255).
//
// Bound by the memory: two lanes take a block of 32, each 16 numbers, so that a
// lane's loads and its store of codes are 16 bytes wide (8 of E2M1).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "mx_format.cuh"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kShare = 16;  // numbers a thread

template <int kType>
__device__ __forceinline__ void load_share(const void* base, int64_t element, float (&v)[kShare]) {
  if constexpr (kType == MXFP8_FP32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + element);
#pragma unroll
    for (int i = 0; i < kShare / 4; ++i) {
      const float4 f = p[i];
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + element);
#pragma unroll
    for (int i = 0; i < kShare / 8; ++i) {
      const uint4 u = p[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kType == MXFP8_BF16) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          v[8 * i + 2 * j] = f.x, v[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
  }
}

template <int kType, int kBits>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ QuantizeParams p) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const uint32_t i = blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x;
  const uint32_t per_row = static_cast<uint32_t>(p.k) / kShare;
  const uint32_t row = i / per_row, at = (i - row * per_row) * kShare;
  // Both lanes of a block take the same way: a block's two shares are one row's.
  int64_t from = row;
  bool live = i < p.items;
  if (live && p.rows) {
    from = p.rows[row];
    if (from < 0 || from >= p.x_rows) {
      if (from != -1 && p.flags) atomicOr(p.flags, MXFP8_FLAG_BAD_INDEX);
      live = false;
    }
  }
  float v[kShare];
#pragma unroll
  for (int j = 0; j < kShare; ++j) v[j] = 0.0f;
  if (live) load_share<kType>(p.x, from * p.x_stride + at, v);
  // Magnitudes as integers keep their order, and what is not finite lies above.
  uint32_t top = 0u;
  bool finite = true;
#pragma unroll
  for (int j = 0; j < kShare; ++j) {
    const uint32_t m = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    if (m < 0x7F800000u) {
      top = max(top, m);
    } else {
      finite = false;
      v[j] = __uint_as_float(0x7FC00000u);
    }
  }
  top = max(top, __shfl_xor_sync(~0u, top, 1));
  if constexpr (kBits == 4) finite = __shfl_xor_sync(~0u, finite, 1) && finite;
  if (!live) return;
  const size_t block = static_cast<size_t>(i) / 2;
  if constexpr (kBits == 8) {
    const uint32_t code = scale_code(__uint_as_float(top));
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = to_e4m3(v[4 * j], v[4 * j + 1], code) |
             to_e4m3(v[4 * j + 2], v[4 * j + 3], code) << 16;
    *reinterpret_cast<uint4*>(p.codes + static_cast<size_t>(i) * kShare) =
        make_uint4(w[0], w[1], w[2], w[3]);
    if (i % 2 == 0) p.scales[block] = static_cast<uint8_t>(code);
  } else {
    const uint32_t code = scale_code_e2m1(__uint_as_float(top));
    uint32_t w[2] = {0u, 0u};
    if (finite)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j / 4] |= to_e2m1(v[2 * j], v[2 * j + 1], code) << (8 * (j % 4));
    *reinterpret_cast<uint2*>(p.codes + static_cast<size_t>(i) * (kShare / 2)) =
        make_uint2(w[0], w[1]);
    if (i % 2 == 0) p.scales[block] = static_cast<uint8_t>(finite ? code : 255u);
  }
}

// Values of 16 numbers: exact in FP32; rounded once where the type is narrower
// than a value's exponent.
template <int kType, int kBits>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* out, uint32_t items) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const uint32_t i = blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x;
  if (i >= items) return;
  const size_t first = static_cast<size_t>(i) * kShare;
  const uint32_t code = scales[i / 2];
  // 2^(code - 127) as two exact factors; NaN for the code 255.
  const int e = static_cast<int>(code) - 127;
  const float s = code == 255u ? __uint_as_float(0x7FC00000u)
                               : __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
  const float r = __uint_as_float(static_cast<uint32_t>(127 + (code == 255u ? 0 : e - e / 2)) << 23);
  float2 v[kShare / 2];
  if constexpr (kBits == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(codes + first);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w[j / 2] >> (16 * (j % 2))), __NV_E4M3);
      v[j] = __half22float2(__half2(h));
    }
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(codes + first / 2);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
          static_cast<__nv_fp4x2_storage_t>(w[j / 4] >> (8 * (j % 4))), __NV_E2M1);
      v[j] = __half22float2(__half2(h));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = make_float2(v[j].x * s * r, v[j].y * s * r);
  if constexpr (kType == MXFP8_FP32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + first);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (kType == MXFP8_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[j].x, v[j].y);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 h = __floats2half2_rn(v[j].x, v[j].y);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + first);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), uint32_t items, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3((items + kThreads - 1) / kThreads);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int kBits>
cudaError_t quantize_as(const QuantizeParams& p, cudaStream_t stream) {
  switch (p.type) {
    case MXFP8_BF16: return launch(quantize_kernel<MXFP8_BF16, kBits>, p.items, stream, p);
    case MXFP8_FP16: return launch(quantize_kernel<MXFP8_FP16, kBits>, p.items, stream, p);
    default: return launch(quantize_kernel<MXFP8_FP32, kBits>, p.items, stream, p);
  }
}
template <int kBits>
cudaError_t dequantize_as(const uint8_t* codes, const uint8_t* scales, void* out, int type,
                          uint32_t items, cudaStream_t stream) {
  switch (type) {
    case MXFP8_BF16:
      return launch(dequantize_kernel<MXFP8_BF16, kBits>, items, stream, codes, scales, out, items);
    case MXFP8_FP16:
      return launch(dequantize_kernel<MXFP8_FP16, kBits>, items, stream, codes, scales, out, items);
    default:
      return launch(dequantize_kernel<MXFP8_FP32, kBits>, items, stream, codes, scales, out, items);
  }
}

}  // namespace

cudaError_t launch_quantize(const QuantizeParams& p, cudaStream_t stream) {
  return p.format == MXFP8_FORMAT_MXFP8 ? quantize_as<8>(p, stream) : quantize_as<4>(p, stream);
}
cudaError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, void* out, int format,
                              int type, uint32_t items, cudaStream_t stream) {
  return format == MXFP8_FORMAT_MXFP8
             ? dequantize_as<8>(codes, scales, out, type, items, stream)
             : dequantize_as<4>(codes, scales, out, type, items, stream);
}

}  // namespace mxfp8
