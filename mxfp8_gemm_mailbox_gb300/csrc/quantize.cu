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
// Bound by the memory: two lanes take a block of 32, each 16 numbers (a 32-byte sector of
// 16-bit ones), twice, so that 64 bytes a thread are under way; the largest magnitude of
// 16-bit numbers is found two at a time and a scale is one factor, which leaves some four
// instructions a number (with a comparison and two factors each the arithmetic took longer
// than the memory: 139 us below).
//
// Measured: 16384 x 8192 BF16 to MXFP4 and back 103 us for 687 MB, 6.7 TB/s (the copy rate is
// 6.78); one share a thread 106, four 105.  64 gathered rows of 7168: 1.7 us, the launch and
// two round trips.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "mx_format.cuh"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kShare = 16;  // numbers a thread takes at a time
constexpr int kItems = 2;   // times

// A share as it lies in memory, 32 bytes of 16-bit numbers or 64 of FP32, and its values.
template <int kType>
struct Share {
  static constexpr int kWords = kType == MXFP8_FP32 ? 16 : 8;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* base, int64_t element, bool sectors) {
    const uint32_t* const p = kType == MXFP8_FP32
                                  ? static_cast<const uint32_t*>(base) + element
                                  : reinterpret_cast<const uint32_t*>(
                                        static_cast<const uint16_t*>(base) + element);
#pragma unroll
    for (int i = 0; i < kWords; i += 8) {
      if (sectors) {
        uint32_t r[8];
        ptx::ld_once_v8(p + i, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i + j] = r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const uint4 u = ptx::ld_once_v4(p + i + j);
          w[i + j] = u.x, w[i + j + 1] = u.y, w[i + j + 2] = u.z, w[i + j + 3] = u.w;
        }
      }
    }
  }
  // The largest magnitude's bits in FP32, where nothing is infinite or NaN; else at
  // least infinity's.  (Magnitudes as integers keep their order; 16-bit ones go two at a
  // time.)
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0u;
    if constexpr (kType == MXFP8_FP32) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      if constexpr (kType == MXFP8_BF16) return m << 16;
      return m >= 0x7C00u ? 0x7F800000u
                          : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
    }
  }
  __device__ __forceinline__ void values(float (&v)[kShare]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kType == MXFP8_FP32) {
        v[i] = __uint_as_float(w[i]);
      } else if constexpr (kType == MXFP8_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
    }
  }
};

template <int kType, int kBits>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ QuantizeParams p) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const uint32_t first = blockIdx.x * static_cast<uint32_t>(kThreads * kItems) + threadIdx.x;
  const uint32_t per_row = static_cast<uint32_t>(p.k) / kShare;
  Share<kType> share[kItems];
  bool live[kItems];
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    // Both lanes of a block take the same way: a block's two shares are one row's.
    const uint32_t i = first + n * kThreads;
    live[n] = i < p.items;
    if (!live[n]) continue;
    const uint32_t row = i / per_row;
    const int64_t at = static_cast<int64_t>(i - row * per_row) * kShare;
    int64_t from = row;
    if (p.rows) {
      from = p.rows[from];
      if (from < 0 || from >= p.x_rows) {
        if (from != -1 && p.flags) atomicOr(p.flags, MXFP8_FLAG_BAD_INDEX);
        live[n] = false;
        continue;
      }
    }
    share[n].load(p.x, from * p.x_stride + at, p.sectors);
  }
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const uint32_t i = first + n * kThreads;
    float v[kShare];
    uint32_t top = 0u;
    if (live[n]) {
      share[n].values(v);
      top = share[n].top();
    }
    bool finite = top < 0x7F800000u;
    if constexpr (kBits == 4) finite = __shfl_xor_sync(~0u, finite, 1) && finite;
    if (!finite && kBits == 8) {  // the scale is that of the finite ones
      top = 0u;
#pragma unroll
      for (int j = 0; j < kShare; ++j) {
        const uint32_t m = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        if (m < 0x7F800000u)
          top = max(top, m);
        else
          v[j] = __uint_as_float(0x7FC00000u);
      }
    }
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    if (!live[n]) continue;
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
}

// Values of 16 numbers: exact in FP32 below 2^128, infinite from there on; rounded once
// where the type is narrower than a value's exponent.
template <int kType, int kBits>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* out, uint32_t items) {
  constexpr int kWords = kBits / 2;  // of a share's codes
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const uint32_t first = blockIdx.x * static_cast<uint32_t>(kThreads * kItems) + threadIdx.x;
  uint32_t w[kItems][kWords], code[kItems];
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const uint32_t i = first + n * kThreads;
    if (i >= items) continue;
    code[n] = scales[i / 2];
    const uint8_t* const from = codes + static_cast<size_t>(i) * kShare * kBits / 8;
    if constexpr (kBits == 8) {
      const uint4 u = ptx::ld_once_v4(from);
      w[n][0] = u.x, w[n][1] = u.y, w[n][2] = u.z, w[n][3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(from);
      w[n][0] = u.x, w[n][1] = u.y;
    }
  }
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const uint32_t i = first + n * kThreads;
    if (i >= items) continue;
    const float s = scale_of(code[n]);
    float2 v[kShare / 2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (kBits == 8) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(w[n][j / 2] >> (16 * (j % 2))), __NV_E4M3);
        v[j] = __half22float2(__half2(h));
      } else {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
            static_cast<__nv_fp4x2_storage_t>(w[n][j / 4] >> (8 * (j % 4))), __NV_E2M1);
        v[j] = __half22float2(__half2(h));
      }
      v[j] = make_float2(v[j].x * s, v[j].y * s);
    }
    const size_t to = static_cast<size_t>(i) * kShare;
    if constexpr (kType == MXFP8_FP32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
    } else {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kType == MXFP8_BF16) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[j].x, v[j].y);
          u[j] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
          const __half2 h = __floats2half2_rn(v[j].x, v[j].y);
          u[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      uint16_t* const o = static_cast<uint16_t*>(out) + to;
      if (reinterpret_cast<uintptr_t>(out) % 32 == 0) {
        ptx::st_v8(o, u);
      } else {
        ptx::st_v4(o, make_uint4(u[0], u[1], u[2], u[3]));
        ptx::st_v4(o + 8, make_uint4(u[4], u[5], u[6], u[7]));
      }
    }
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
  constexpr uint32_t kEach = kThreads * kItems;
  cfg.gridDim = dim3(items / kEach + (items % kEach ? 1 : 0));
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
