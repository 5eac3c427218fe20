// The products that lead into and out of the latent space, one matrix a head:
//
//   query:  q[t][h][c] = sum_d W[h][c][d] q_nope[t][h][d], the rotary part
//           copied behind it (BF16);
//   values: y[t][h][v] = sum_c W[h][v][c] o[t][h][c], rounded to MXFP8 along
//           the row [h][v] in blocks of 32, which is the projection's x.
//
// Sums in FP32.  A block's scale is the smallest power of two under which no
// element passes 448, E4M3's largest, so none saturates; the elements are
// rounded to nearest, ties to even.  An element that is not finite is NaN and
// no part of its block's scale.
//
// Few rows against many matrices: bound by reading W once (16.8 MB at 128
// heads, 512 x 128).  A warp owns 32 outputs of one head and holds their rows
// of W in registers as the A operand of m16n8k16 products, the up to 8 rows of
// activations (16 rows the A tile's, 8 the B tile's) being B: the tensor core
// does the widening and the sums, one 16-byte load a lane feeds two products,
// and every byte of W is read by one lane once.  The order of a product's inner
// indexes is free, so lane (g, q) loads 8 consecutive numbers of row g at
// 32 k + 8 q for both operands, and the products take them as they lie.  Long
// sums are cut over two or four warps of a block (128 numbers a warp where that
// divides them), so that every weight a warp needs is on its way at once, before
// the wait for the kernel that makes the activations.  (The legacy product
// instruction suffices: 8 rows are 3 % of the tensor cores' time.)
//
// Measured, 8 rows and 128 heads, one call after another: query 128 -> 512 3.6
// us = 5.2 TB/s (19 MB), values 512 -> 128 4.1 us = 4.4 TB/s (18 MB); 1 row,
// 16 and 32 heads: 1.4 and 2.2 us, launch and two round trips to memory.
#include <cuda_bf16.h>

#include "internal.h"
#include "mx_format.cuh"
#include "ptx.cuh"

namespace mxfp8 {
namespace {

constexpr int kRope = 64;
constexpr int kRowsPerBlock = 8;  // the B operand's columns

// D (16 x 8, FP32) += A (16 x 16) B (16 x 8), BF16.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Warps that share an output's sum over `inner` numbers.
__host__ __device__ constexpr int sum_warps(int inner) {
  const int steps = inner / 32;
  return steps > 8 && steps % 4 == 0 ? 4 : steps > 4 && steps % 2 == 0 ? 2 : 1;
}

// The sums over kCount numbers of 32 outputs (rows of w, kInner apart) for up
// to 8 rows of activations: acc[0] holds outputs 0 .. 15, acc[1] the next 16;
// element e of lane (g, q) is output g + 8 (e / 2), row 2 q + e % 2.  Products
// of even and odd halves of a load go to two accumulators, so the longest
// chain of dependent sums is halved.
template <int kInner, int kCount>
__device__ __forceinline__ void products(const uint16_t* __restrict__ w,
                                         const uint16_t* __restrict__ in, size_t in_stride,
                                         int rows, float (&acc)[2][4]) {
  constexpr int kSteps = kCount / 32;
  constexpr int kBatch = kSteps < 8 ? kSteps : 8;  // loads in flight a lane and row
  const int g = threadIdx.x % 32 / 4, q = threadIdx.x % 4;
  float part[2][2][4] = {};
  const uint16_t* wp = w + static_cast<size_t>(g) * kInner + q * 8;
  const bool live = g < rows;
  const uint16_t* ip = in + (live ? g : 0) * in_stride + q * 8;
#pragma unroll
  for (int k0 = 0; k0 < kSteps; k0 += kBatch) {
    uint4 a[4][kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k < kSteps)
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r][k] = ptx::ld_once_v4(wp + r * 8 * kInner + (k0 + k) * 32);
    // The weights do not depend on the kernel before; the activations do.
    if (k0 == 0) ptx::grid_dependency_wait();
    uint4 b[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      b[k] = make_uint4(0u, 0u, 0u, 0u);
      if (k0 + k < kSteps && live) b[k] = *reinterpret_cast<const uint4*>(ip + (k0 + k) * 32);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k0 + k >= kSteps) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        mma_16816(part[half][0], a[2 * half][k].x, a[2 * half + 1][k].x, a[2 * half][k].y,
                  a[2 * half + 1][k].y, b[k].x, b[k].y);
        mma_16816(part[half][1], a[2 * half][k].z, a[2 * half + 1][k].z, a[2 * half][k].w,
                  a[2 * half + 1][k].w, b[k].z, b[k].w);
      }
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[half][e] = part[half][0][e] + part[half][1][e];
}

struct ProjectParams {
  const uint16_t* in;    // [rows][heads][inner]
  const uint16_t* rope;  // query: [rows][heads][64]
  const uint16_t* w;     // [heads][outer][inner]
  uint16_t* q;           // query: [rows][heads][outer + 64]
  uint8_t* x;            // values: [rows][heads x outer]
  uint8_t* x_scale;      // values: [rows][heads x outer / 32]
  int rows, heads, outer;
};

constexpr int kWarps = 4;  // of a block

// kShare warps take 32 outputs of one head (for the query, one piece more a
// head is the rotary part); grid.y = groups of 8 rows.
template <bool kQuery, int kInner>
__global__ void __launch_bounds__(32 * kWarps)
    project_kernel(const __grid_constant__ ProjectParams p) {
  constexpr int kShare = sum_warps(kInner);
  __shared__ float4 sums[kWarps][2][32];
  ptx::launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int pieces = p.outer / 32 + (kQuery ? 1 : 0);  // of a head
  const int piece = blockIdx.x * (kWarps / kShare) + warp / kShare, slice = warp % kShare;
  const int h = piece / pieces, at = piece % pieces;
  const int t0 = blockIdx.y * kRowsPerBlock, rows = min(kRowsPerBlock, p.rows - t0);
  const bool copies = kQuery && at == pieces - 1;
  const int j0 = at * 32;
  float acc[2][4] = {};
  if (h < p.heads && !copies)
    products<kInner, kInner / kShare>(
        p.w + (static_cast<size_t>(h) * p.outer + j0) * kInner + slice * (kInner / kShare),
        p.in + (static_cast<size_t>(t0) * p.heads + h) * kInner + slice * (kInner / kShare),
        static_cast<size_t>(p.heads) * kInner, rows, acc);
  if constexpr (kShare > 1) {
    if (slice > 0)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        sums[warp][half][lane] =
            make_float4(acc[half][0], acc[half][1], acc[half][2], acc[half][3]);
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int other = 1; other < kShare; ++other)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float4 v = sums[warp + other][half][lane];
        acc[half][0] += v.x, acc[half][1] += v.y, acc[half][2] += v.z, acc[half][3] += v.w;
      }
  }
  if (h >= p.heads) return;
  if (copies) {
    if (slice > 0) return;
    ptx::grid_dependency_wait();
    for (int i = lane; i < rows * (kRope / 8); i += 32) {
      const size_t th = static_cast<size_t>(t0 + i / (kRope / 8)) * p.heads + h;
      const int c = i % (kRope / 8) * 8;
      *reinterpret_cast<uint4*>(p.q + th * (p.outer + kRope) + p.outer + c) =
          *reinterpret_cast<const uint4*>(p.rope + th * kRope + c);
    }
    return;
  }
  if constexpr (kQuery) {
    // Neighbouring outputs lie in lanes 4 apart: pairs of lanes exchange, and
    // the even one of each pair writes two outputs of its row 2 q, the odd one
    // of row 2 q + 1.
    const bool odd = g & 1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int half = e / 2, up = e % 2;
      const float send = odd ? acc[half][2 * up] : acc[half][2 * up + 1];
      const float got = __shfl_xor_sync(~0u, send, 4);
      const float lo = odd ? got : acc[half][2 * up], hi = odd ? acc[half][2 * up + 1] : got;
      const int t = 2 * q + (odd ? 1 : 0);
      if (t < rows) {
        const size_t th = static_cast<size_t>(t0 + t) * p.heads + h;
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        *reinterpret_cast<__nv_bfloat162*>(p.q + th * (p.outer + kRope) + j0 + half * 16 + up * 8 +
                                           (g & ~1)) = v;
      }
    }
  } else {
    // An infinity has no E4M3 code, and the conversion would make 448 of it.
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!isfinite(acc[half][e])) acc[half][e] = __uint_as_float(0x7FC00000u);
    // One scale block is a warp's 32 outputs of a row: its largest magnitude
    // over the lanes of equal q.  (fmaxf passes over NaN.)
#pragma unroll
    for (int up = 0; up < 2; ++up) {
      float top = fmaxf(fmaxf(fabsf(acc[0][up]), fabsf(acc[0][2 + up])),
                        fmaxf(fabsf(acc[1][up]), fabsf(acc[1][2 + up])));
      top = fmaxf(top, 0.0f);
#pragma unroll
      for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      const uint32_t code = scale_code(top);
      // Outputs g, g + 8, g + 16, g + 24 of row 2 q + up; four lanes' bytes
      // gather into a word of the first of them.
      const int t = 2 * q + up;
      const size_t block = (static_cast<size_t>(t0 + t) * p.heads + h) * (p.outer / 32) + at;
      const uint32_t low = to_e4m3(acc[0][up], acc[0][2 + up], code);
      const uint32_t high = to_e4m3(acc[1][up], acc[1][2 + up], code);
      uint32_t word[4] = {low & 0xFFu, low >> 8, high & 0xFFu, high >> 8};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        word[i] <<= 8 * (g % 4);
        word[i] |= __shfl_xor_sync(~0u, word[i], 4);
        word[i] |= __shfl_xor_sync(~0u, word[i], 8);
      }
      if (t < rows) {
        if (g == 0) p.x_scale[block] = static_cast<uint8_t>(code);
        if (g % 4 == 0)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint32_t*>(p.x + block * 32 + i * 8 + g) = word[i];
      }
    }
  }
}

template <bool kQuery, int kInner>
cudaError_t launch_impl(const ProjectParams& p, cudaStream_t stream) {
  const int pieces = p.heads * (p.outer / 32 + (kQuery ? 1 : 0));
  constexpr int kPieces = kWarps / sum_warps(kInner);  // of a block
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(32 * kWarps);
  cfg.gridDim = dim3(static_cast<unsigned>((pieces + kPieces - 1) / kPieces),
                     static_cast<unsigned>((p.rows + kRowsPerBlock - 1) / kRowsPerBlock));
  return cudaLaunchKernelEx(&cfg, project_kernel<kQuery, kInner>, p);
}

template <bool kQuery>
cudaError_t launch_for_inner(const ProjectParams& p, int inner, cudaStream_t stream) {
  switch (inner) {
    case 32: return launch_impl<kQuery, 32>(p, stream);
    case 64: return launch_impl<kQuery, 64>(p, stream);
    case 96: return launch_impl<kQuery, 96>(p, stream);
    case 128: return launch_impl<kQuery, 128>(p, stream);
    case 160: return launch_impl<kQuery, 160>(p, stream);
    case 192: return launch_impl<kQuery, 192>(p, stream);
    case 224: return launch_impl<kQuery, 224>(p, stream);
    case 256: return launch_impl<kQuery, 256>(p, stream);
    case 288: return launch_impl<kQuery, 288>(p, stream);
    case 320: return launch_impl<kQuery, 320>(p, stream);
    case 352: return launch_impl<kQuery, 352>(p, stream);
    case 384: return launch_impl<kQuery, 384>(p, stream);
    case 416: return launch_impl<kQuery, 416>(p, stream);
    case 448: return launch_impl<kQuery, 448>(p, stream);
    case 480: return launch_impl<kQuery, 480>(p, stream);
    case 512: return launch_impl<kQuery, 512>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_latent_query(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w,
                                uint16_t* q, int rows, int heads, int nope, int latent,
                                cudaStream_t stream) {
  const ProjectParams p{q_nope, q_rope, w, q, nullptr, nullptr, rows, heads, latent};
  return launch_for_inner<true>(p, nope, stream);
}

cudaError_t launch_latent_values(const uint16_t* o, const uint16_t* w, uint8_t* x,
                                 uint8_t* x_scale, int rows, int heads, int latent, int value,
                                 cudaStream_t stream) {
  const ProjectParams p{o, nullptr, w, nullptr, x, x_scale, rows, heads, value};
  return latent == 512 ? launch_impl<false, 512>(p, stream) : launch_impl<false, 256>(p, stream);
}

}  // namespace mxfp8
