// The latent-attention calls of include/mxfp8_mailbox.h: argument checks and
// launches.  Every check happens on the host before a launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "internal.h"

using namespace mxfp8;

namespace {

mxfp8_status check_heads(int32_t rows, int32_t heads, int32_t latent) {
  if (rows < 0) return fail(MXFP8_ERR_INVALID, "rows must not be negative");
  if (heads < 1 || heads > MXFP8_MAX_HEADS)
    return fail(MXFP8_ERR_UNSUPPORTED, "heads must be in 1.." + std::to_string(MXFP8_MAX_HEADS) +
                                           ", got " + std::to_string(heads));
  if (rows > MXFP8_MAX_LATENT_ROWS)
    return fail(MXFP8_ERR_UNSUPPORTED, "rows must be at most " +
                                           std::to_string(MXFP8_MAX_LATENT_ROWS) + ", got " +
                                           std::to_string(rows));
  if (latent != 256 && latent != 512)
    return fail(MXFP8_ERR_UNSUPPORTED, "latent must be 256 or 512, got " + std::to_string(latent));
  return MXFP8_OK;
}

mxfp8_status check_width(const char* name, int32_t width) {
  if (width < 32 || width > 512 || width % 32)
    return fail(MXFP8_ERR_UNSUPPORTED, std::string(name) +
                                           " must be a multiple of 32 in 32..512, got " +
                                           std::to_string(width));
  return MXFP8_OK;
}

mxfp8_status check_pointer(const char* name, const void* p, size_t alignment) {
  if (!p || !aligned(p, alignment))
    return fail(MXFP8_ERR_INVALID, std::string(name) + " must be a " + std::to_string(alignment) +
                                       "-byte aligned device pointer");
  return MXFP8_OK;
}

}  // namespace

#define CHECK(expr)                                \
  do {                                             \
    const mxfp8_status checked = (expr);           \
    if (checked != MXFP8_OK) return checked;       \
  } while (0)

extern "C" {

mxfp8_status mxfp8_latent_query(const void* q_nope, const void* q_rope, const void* w, void* q,
                                int32_t rows, int32_t heads, int32_t nope, int32_t latent,
                                void* stream) {
  CHECK(check_heads(rows, heads, latent));
  CHECK(check_width("nope", nope));
  if (rows == 0) return MXFP8_OK;
  CHECK(check_pointer("q_nope", q_nope, 16));
  CHECK(check_pointer("q_rope", q_rope, 16));
  CHECK(check_pointer("w", w, 16));
  CHECK(check_pointer("q", q, 16));
  const cudaError_t e = launch_latent_query(
      static_cast<const uint16_t*>(q_nope), static_cast<const uint16_t*>(q_rope),
      static_cast<const uint16_t*>(w), static_cast<uint16_t*>(q), rows, heads, nope, latent,
      static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the latent queries");
  return MXFP8_OK;
}

mxfp8_status mxfp8_latent_values(const void* o, const void* w, void* x, void* x_scale,
                                 int32_t rows, int32_t heads, int32_t latent, int32_t value,
                                 void* stream) {
  CHECK(check_heads(rows, heads, latent));
  CHECK(check_width("value", value));
  if (rows == 0) return MXFP8_OK;
  CHECK(check_pointer("o", o, 16));
  CHECK(check_pointer("w", w, 16));
  CHECK(check_pointer("x", x, 16));
  CHECK(check_pointer("x_scale", x_scale, 1));
  const cudaError_t e = launch_latent_values(
      static_cast<const uint16_t*>(o), static_cast<const uint16_t*>(w), static_cast<uint8_t*>(x),
      static_cast<uint8_t*>(x_scale), rows, heads, latent, value,
      static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the latent values");
  return MXFP8_OK;
}

size_t mxfp8_latent_workspace_bytes(int32_t latent) {
  if (latent != 256 && latent != 512) return 0;
  return latent_workspace_bytes(latent);
}

mxfp8_status mxfp8_latent_attend(const mxfp8_latent_desc* d, const void* q, const void* cache,
                                 const int32_t* page_table, const int32_t* lengths,
                                 const int32_t* row_begin, const int64_t* tree, void* out,
                                 void* workspace, size_t workspace_bytes, int32_t* flags,
                                 void* stream) {
  if (!d) return fail(MXFP8_ERR_INVALID, "desc is NULL");
  CHECK(check_heads(d->rows, d->heads, d->latent));
  const int64_t width = d->latent + MXFP8_LATENT_ROPE;
  if (d->requests < 0 || d->requests > MXFP8_MAX_REQUESTS)
    return fail(MXFP8_ERR_UNSUPPORTED, "requests must be in 0.." +
                                           std::to_string(MXFP8_MAX_REQUESTS) + ", got " +
                                           std::to_string(d->requests));
  if (d->page_size < 8 || d->page_size % 8)
    return fail(MXFP8_ERR_UNSUPPORTED, "page_size must be a positive multiple of 8, got " +
                                           std::to_string(d->page_size));
  if (d->pages < 1 || d->table_width < 1)
    return fail(MXFP8_ERR_INVALID, "pages and table_width must be positive");
  if (static_cast<int64_t>(d->table_width) * d->page_size > INT32_MAX - 128)
    return fail(MXFP8_ERR_UNSUPPORTED, "a page table spans at most 2^31 - 129 tokens");
  // Token tiles of all row tiles at most (64 tokens, 128 rows), numbered in 31 bits.
  if ((static_cast<int64_t>(d->rows) * d->heads / 128 + d->requests) *
          ((static_cast<int64_t>(d->table_width) * d->page_size + 63) / 64) >
      1 << 30)
    return fail(MXFP8_ERR_UNSUPPORTED, "rows x heads x tokens is past 2^30 tiles of 128 x 64");
  if (d->token_stride < width || d->token_stride % 8 || d->page_stride % 8 ||
      (d->pages > 1 && d->page_stride < width))
    return fail(MXFP8_ERR_UNSUPPORTED,
                "the cache's strides must be multiples of 8 elements and at least a token's width");
  if (!(d->scale > 0.0f) || !std::isfinite(d->scale))
    return fail(MXFP8_ERR_INVALID, "scale must be positive and finite");
  if (d->rows == 0) return MXFP8_OK;
  if (d->requests == 0) return fail(MXFP8_ERR_INVALID, "query rows without a request");
  CHECK(check_pointer("q", q, 16));
  CHECK(check_pointer("cache", cache, 16));
  CHECK(check_pointer("page_table", page_table, 4));
  CHECK(check_pointer("lengths", lengths, 4));
  CHECK(check_pointer("row_begin", row_begin, 4));
  if (tree) CHECK(check_pointer("tree", tree, 8));
  CHECK(check_pointer("out", out, 16));
  CHECK(check_pointer("workspace", workspace, 256));
  if (workspace_bytes < mxfp8_latent_workspace_bytes(d->latent))
    return fail(MXFP8_ERR_INVALID,
                "the workspace must hold " +
                    std::to_string(mxfp8_latent_workspace_bytes(d->latent)) + " bytes");
  if (flags) CHECK(check_pointer("flags", flags, 4));
  LatentParams p{};
  p.heads = d->heads;
  p.rows = d->rows;
  p.requests = d->requests;
  p.page_size = d->page_size;
  p.pages = d->pages;
  p.table_width = d->table_width;
  p.token_stride = d->token_stride;
  p.page_stride = d->page_stride;
  // Finite still where the product with log2(e) is not: a difference of scores is then
  // past what the exponential takes either way, and equal ones stay equal.
  p.scale_log2 = static_cast<float>(
      std::min(static_cast<double>(d->scale) * 1.4426950408889634,
               static_cast<double>(std::numeric_limits<float>::max())));
  p.q = static_cast<const uint16_t*>(q);
  p.cache = static_cast<const uint16_t*>(cache);
  p.table = page_table;
  p.lengths = lengths;
  p.row_begin = row_begin;
  p.tree = tree;
  p.out = static_cast<uint16_t*>(out);
  p.flags = flags;
  const cudaError_t e = launch_latent_attend(p, d->latent, workspace, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the latent attention");
  return MXFP8_OK;
}

}  // extern "C"
