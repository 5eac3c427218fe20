// The calls of a layer of routed experts of include/mxfp8_mailbox.h: argument
// checks and launches.  Every check happens on the host before a launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

using namespace mxfp8;

namespace {

mxfp8_status check_pointer(const char* name, const void* p, size_t alignment) {
  if (!p || !aligned(p, alignment))
    return fail(MXFP8_ERR_INVALID, std::string(name) + " must be a " + std::to_string(alignment) +
                                       "-byte aligned device pointer");
  return MXFP8_OK;
}
mxfp8_status check_type(int32_t type) {
  if (type != MXFP8_BF16 && type != MXFP8_FP16 && type != MXFP8_FP32)
    return fail(MXFP8_ERR_INVALID, "type must be MXFP8_BF16, MXFP8_FP16 or MXFP8_FP32");
  return MXFP8_OK;
}
mxfp8_status check_codes(const char* name, int32_t format) {
  if (format != MXFP8_FORMAT_MXFP8 && format != MXFP8_FORMAT_MXFP4)
    return fail(MXFP8_ERR_INVALID,
                std::string(name) + " must be MXFP8_FORMAT_MXFP8 or MXFP8_FORMAT_MXFP4");
  return MXFP8_OK;
}

#define CHECK(expr)                                \
  do {                                             \
    const mxfp8_status checked = (expr);           \
    if (checked != MXFP8_OK) return checked;       \
  } while (0)

// What the matrices alone say.
mxfp8_status check_matrices(const mxfp8_expert_desc* d) {
  if (!d) return fail(MXFP8_ERR_INVALID, "desc is NULL");
  if (d->experts < 1 || d->experts > MXFP8_MAX_EXPERTS)
    return fail(MXFP8_ERR_UNSUPPORTED, "experts must be in 1.." +
                                           std::to_string(MXFP8_MAX_EXPERTS) + ", got " +
                                           std::to_string(d->experts));
  if (d->gated != 0 && d->gated != 1) return fail(MXFP8_ERR_INVALID, "gated must be 0 or 1");
  const int step = d->gated ? 32 : 8;
  if (d->n < step || d->n % step || d->n > 1 << 20)
    return fail(MXFP8_ERR_UNSUPPORTED, "n must be a multiple of " + std::to_string(step) +
                                           " up to 2^20, got " + std::to_string(d->n));
  if (d->k < 128 || d->k % 128 || d->k > 1 << 20)
    return fail(MXFP8_ERR_UNSUPPORTED,
                "k must be a multiple of 128 up to 2^20, got " + std::to_string(d->k));
  if (static_cast<int64_t>(d->experts) * ((d->n + 63) / 64) * d->k > INT32_MAX)
    return fail(MXFP8_ERR_UNSUPPORTED, "experts x n x k is past 2^37");
  return check_codes("w_format", d->w_format);
}
int w_tiles(const mxfp8_expert_desc& d) {
  const int outputs = d.gated ? 64 : 128;  // of a tile
  return (d.n + outputs - 1) / outputs;
}

int row_bytes(int32_t format, int32_t k) { return format == MXFP8_FORMAT_MXFP4 ? k / 2 : k; }

// An axis of a tensor map past the first: its size, how far apart its elements lie in
// bytes, and how many a copy takes.
struct Axis {
  int64_t size, stride;
  int box;
};
// Codes of 8 bits, or of 4, which land as 16 in 16 bytes; a copy takes 128 along the first
// axis.
template <int kAxes>
mxfp8_status encode_codes(CUtensorMap* map, const void* base, int32_t format, int64_t width,
                          const Axis (&axes)[kAxes]) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return fail(MXFP8_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[kAxes + 1], strides[kAxes];
  cuuint32_t box[kAxes + 1], elem[kAxes + 1];
  dims[0] = static_cast<cuuint64_t>(width);
  box[0] = 128;
  for (int i = 0; i < kAxes; ++i) {
    dims[i + 1] = static_cast<cuuint64_t>(axes[i].size);
    strides[i] = static_cast<cuuint64_t>(axes[i].stride);
    box[i + 1] = static_cast<cuuint32_t>(axes[i].box);
  }
  for (cuuint32_t& e : elem) e = 1;
  const CUresult r = fn(
      map,
      format == MXFP8_FORMAT_MXFP4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B
                                   : CU_TENSOR_MAP_DATA_TYPE_UINT8,
      kAxes + 1, const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MXFP8_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(r));
  return MXFP8_OK;
}
// A tile of W along k_tiles k tiles: 128 rows of an expert; gated 32 rows of the gate, theirs
// of the up half, twice.  Gated, blocks of 32 rows are numbered through all experts, and the
// halves lie n rows apart (the last expert's up blocks are reached as the other half of its
// gate's, so that axis ends before them).
mxfp8_status encode_w(CUtensorMap* map, const void* w, const mxfp8_expert_desc& d, int k_tiles) {
  const int64_t row = row_bytes(d.w_format, d.k), n = d.n;
  const Axis k{d.k / 128, row_bytes(d.w_format, 128), k_tiles};
  if (d.gated)
    return encode_codes(map, w, d.w_format, 128,
                        {{32, row, 32},
                         {2, n * row, 2},
                         {(static_cast<int64_t>(d.experts) * 2 - 1) * (n / 32), 32 * row, 2},
                         k});
  return encode_codes(map, w, d.w_format, 128,
                      {{n, row, 128}, {1, n * row, 1}, {d.experts, n * row, 1}, k});
}
// x's rows; the k tiles of more than one a copy are planes.
mxfp8_status encode_x(CUtensorMap* map, const void* x, const mxfp8_expert_desc& d, int rows,
                      int k_tiles) {
  const int64_t row = row_bytes(d.x_format, d.k);
  if (k_tiles == 1)
    return encode_codes(map, x, d.x_format, d.k, {{d.rows, row, rows}, {1, row * d.rows, 1}});
  return encode_codes(map, x, d.x_format, 128,
                      {{d.rows, row, rows}, {d.k / 128, row_bytes(d.x_format, 128), k_tiles}});
}

}  // namespace

extern "C" {

size_t mxfp8_route_workspace_bytes(int64_t tokens, int32_t experts) {
  if (tokens <= kRouteFew || experts < 1 || experts > MXFP8_MAX_EXPERTS || tokens > INT32_MAX)
    return 0;
  const int64_t block = route_block_tokens(tokens);
  return static_cast<size_t>((tokens + block - 1) / block + 1) * experts * 4;
}

mxfp8_status mxfp8_route(const void* logits, int32_t type, int64_t stride, int64_t tokens,
                         int32_t experts, int32_t k, int32_t normalize, float* weight,
                         int32_t* expert, int32_t* slot, int32_t* row, int32_t* begin,
                         void* workspace, size_t workspace_bytes, void* stream) {
  CHECK(check_type(type));
  if (experts < 1 || experts > MXFP8_MAX_EXPERTS)
    return fail(MXFP8_ERR_UNSUPPORTED, "experts must be in 1.." +
                                           std::to_string(MXFP8_MAX_EXPERTS) + ", got " +
                                           std::to_string(experts));
  if (k < 1 || k > std::min(experts, MXFP8_MAX_CHOICES))
    return fail(MXFP8_ERR_UNSUPPORTED, "k must be in 1.." +
                                           std::to_string(std::min(experts, MXFP8_MAX_CHOICES)) +
                                           ", got " + std::to_string(k));
  if (tokens < 0) return fail(MXFP8_ERR_INVALID, "tokens must not be negative");
  if (tokens > INT32_MAX / k)
    return fail(MXFP8_ERR_UNSUPPORTED, "tokens x k must be below 2^31");
  if (stride < experts && tokens > 1)
    return fail(MXFP8_ERR_INVALID, "stride must be at least experts");
  CHECK(check_pointer("begin", begin, 4));
  const size_t need = mxfp8_route_workspace_bytes(tokens, experts);
  if (tokens > 0) {
    CHECK(check_pointer("logits", logits, type == MXFP8_FP32 ? 4 : 2));
    CHECK(check_pointer("weight", weight, 4));
    CHECK(check_pointer("expert", expert, 4));
    CHECK(check_pointer("slot", slot, 4));
    CHECK(check_pointer("row", row, 4));
  }
  if (need > 0) {
    CHECK(check_pointer("workspace", workspace, 4));
    if (workspace_bytes < need)
      return fail(MXFP8_ERR_INVALID,
                  "the workspace must hold " + std::to_string(need) + " bytes");
  }
  const int64_t step = type == MXFP8_FP32 ? 4 : 8;  // elements of 16 bytes
  RouteParams p{};
  p.tokens = tokens;
  p.stride = stride;
  p.block = route_block_tokens(tokens);
  p.experts = experts;
  p.k = k;
  p.type = type;
  p.normalize = normalize ? 1 : 0;
  p.pairs = experts % 2 == 0 && stride % 2 == 0 && aligned(logits, 4);
  p.wide = aligned(logits, 16) && (tokens <= 1 || stride % step == 0);
  p.logits = logits;
  p.weight = weight;
  p.expert = expert;
  p.slot = slot;
  p.row = row;
  p.begin = begin;
  p.counts = static_cast<int32_t*>(workspace);
  const cudaError_t e = launch_route(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the routing");
  return MXFP8_OK;
}

mxfp8_status mxfp8_quantize(const void* x, int32_t type, int64_t stride, int64_t x_rows, int32_t k,
                            const int32_t* rows, int64_t out_rows, int32_t format, void* codes,
                            void* scales, int32_t* flags, void* stream) {
  CHECK(check_type(type));
  CHECK(check_codes("format", format));
  if (k < 32 || k % 32)
    return fail(MXFP8_ERR_UNSUPPORTED,
                "k must be a positive multiple of 32, got " + std::to_string(k));
  if (x_rows < 0 || out_rows < 0) return fail(MXFP8_ERR_INVALID, "rows must not be negative");
  if (!rows && out_rows != x_rows)
    return fail(MXFP8_ERR_INVALID, "without an index there are as many rows out as in");
  const int64_t per_row = k / 16;
  if (out_rows > INT32_MAX / per_row)
    return fail(MXFP8_ERR_UNSUPPORTED, "rows x k is past 2^35");
  if (out_rows == 0) return MXFP8_OK;
  const int64_t step = type == MXFP8_FP32 ? 4 : 8;  // elements of 16 bytes
  if (x_rows > 1 && (stride < k || stride % step))
    return fail(MXFP8_ERR_UNSUPPORTED,
                "the rows' stride must be at least k and a multiple of 16 bytes");
  if (x_rows > 0) CHECK(check_pointer("x", x, 16));
  if (rows) CHECK(check_pointer("rows", rows, 4));
  CHECK(check_pointer("codes", codes, 16));
  CHECK(check_pointer("scales", scales, 1));
  if (flags) CHECK(check_pointer("flags", flags, 4));
  QuantizeParams p{};
  p.format = format;
  p.type = type;
  p.items = static_cast<uint32_t>(out_rows * per_row);
  p.sectors = aligned(x, 32) && (x_rows <= 1 || stride % (2 * step) == 0);
  p.x_rows = x_rows;
  p.x_stride = stride;
  p.k = k;
  p.x = x;
  p.rows = rows;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.flags = flags;
  const cudaError_t e = launch_quantize(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the quantisation");
  return MXFP8_OK;
}

mxfp8_status mxfp8_dequantize(const void* codes, const void* scales, int64_t rows, int32_t k,
                              int32_t format, int32_t type, void* out, void* stream) {
  CHECK(check_type(type));
  CHECK(check_codes("format", format));
  if (k < 32 || k % 32)
    return fail(MXFP8_ERR_UNSUPPORTED,
                "k must be a positive multiple of 32, got " + std::to_string(k));
  if (rows < 0) return fail(MXFP8_ERR_INVALID, "rows must not be negative");
  const int64_t per_row = k / 16;
  if (rows > INT32_MAX / per_row) return fail(MXFP8_ERR_UNSUPPORTED, "rows x k is past 2^35");
  if (rows == 0) return MXFP8_OK;
  CHECK(check_pointer("codes", codes, 16));
  CHECK(check_pointer("scales", scales, 1));
  CHECK(check_pointer("out", out, 16));
  const cudaError_t e = launch_dequantize(
      static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), out, format, type,
      static_cast<uint32_t>(rows * per_row), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the values");
  return MXFP8_OK;
}

size_t mxfp8_expert_scales_bytes(const mxfp8_expert_desc* d) {
  if (check_matrices(d) != MXFP8_OK) return 0;
  return static_cast<size_t>(d->experts) * w_tiles(*d) * (d->k / 128) * 512;
}

mxfp8_status mxfp8_expert_lay_scales(const mxfp8_expert_desc* d, const void* w_scale, void* laid,
                                     void* stream) {
  CHECK(check_matrices(d));
  CHECK(check_pointer("w_scale", w_scale, 4));
  CHECK(check_pointer("laid", laid, 16));
  const cudaError_t e = launch_lay_scales(static_cast<const uint8_t*>(w_scale),
                                          static_cast<uint8_t*>(laid), d->experts, d->n, d->gated,
                                          w_tiles(*d), d->k / 128, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "laying the scales");
  return MXFP8_OK;
}

size_t mxfp8_expert_workspace_bytes(void) {
  return MXFP8_EXPERT_WORKSPACE_ZEROS + expert_partial_bytes(kMaxExpertCtas);
}

mxfp8_status mxfp8_expert_product(const mxfp8_expert_desc* d, const void* w, const void* laid,
                                  const void* x, const void* x_scale, const int32_t* begin,
                                  void* out, void* out_scale, void* workspace,
                                  size_t workspace_bytes, int32_t* flags, void* stream) {
  CHECK(check_matrices(d));
  CHECK(check_codes("x_format", d->x_format));
  const bool codes = d->out_format != MXFP8_FORMAT_BF16;
  if (codes) {
    CHECK(check_codes("out_format", d->out_format));
    if (d->n % 32)
      return fail(MXFP8_ERR_UNSUPPORTED,
                  "n must be a multiple of 32 to be rounded to blocks, got " + std::to_string(d->n));
  }
  if (d->rows < 0) return fail(MXFP8_ERR_INVALID, "rows must not be negative");
  if (!begin && d->experts != 1)
    return fail(MXFP8_ERR_INVALID, "begin is NULL, and there is more than one expert");
  // Rows past the last by a tile's, and by the experts, are still counted in 31 bits.
  if (d->rows > MXFP8_MAX_EXPERT_ROWS)
    return fail(MXFP8_ERR_UNSUPPORTED, "rows must be at most " +
                                           std::to_string(MXFP8_MAX_EXPERT_ROWS) + ", got " +
                                           std::to_string(d->rows));
  // Tiles are numbered in 31 bits (32 rows the smallest).
  if ((static_cast<int64_t>(d->rows) / 32 + d->experts) * w_tiles(*d) > 1 << 30)
    return fail(MXFP8_ERR_UNSUPPORTED, "rows x n is past 2^30 tiles");
  if (d->rows == 0) return MXFP8_OK;
  CHECK(check_pointer("w", w, 32));
  CHECK(check_pointer("laid", laid, 16));
  CHECK(check_pointer("x", x, 32));
  CHECK(check_pointer("x_scale", x_scale, 4));
  if (begin) CHECK(check_pointer("begin", begin, 4));
  CHECK(check_pointer("out", out, 16));
  if (codes) CHECK(check_pointer("out_scale", out_scale, 1));
  CHECK(check_pointer("workspace", workspace, 16));
  if (workspace_bytes < mxfp8_expert_workspace_bytes())
    return fail(MXFP8_ERR_INVALID, "the workspace must hold " +
                                       std::to_string(mxfp8_expert_workspace_bytes()) + " bytes");
  if (flags) CHECK(check_pointer("flags", flags, 4));
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device's SM count");
  const int ctas = std::min(sms, kMaxExpertCtas);
  const ExpertTile tile = expert_tile(d->rows, d->experts, w_tiles(*d), d->k / 128, ctas);
  ExpertMaps maps{};
  CHECK(encode_w(&maps.w, w, *d, tile.k_tiles));
  CHECK(encode_x(&maps.x, x, *d, tile.x_rows, tile.k_tiles));
  CHECK(encode_x(&maps.x_small, x, *d, tile.x_small, tile.k_tiles));
  constexpr uint32_t kE2M1 = 5;  // the products' type codes; E4M3 is 0
  ExpertParams p{};
  p.experts = d->experts;
  p.n = d->n;
  p.rows = d->rows;
  p.w_tiles = w_tiles(*d);
  p.k_tiles = d->k / 128;
  p.gated = d->gated;
  p.format = d->out_format;
  p.idesc = 1u << 23 | (tile.kind == ExpertTile::kWide ? 256u : 128u) >> 4 << 24 |
            (d->w_format == MXFP8_FORMAT_MXFP4 ? kE2M1 << 7 : 0u) |
            (d->x_format == MXFP8_FORMAT_MXFP4 ? kE2M1 << 10 : 0u);
  // A copy counts the bytes that it reads, not the places that 4-bit elements take.
  const uint32_t x_row = tile.k_tiles * (d->x_format == MXFP8_FORMAT_MXFP4 ? 64 : 128);
  p.w_bytes = 128 * tile.k_tiles * (d->w_format == MXFP8_FORMAT_MXFP4 ? 64 : 128);
  p.x_bytes = tile.x_rows * x_row;
  p.x_small_bytes = tile.x_small * x_row;
  p.w_sf = static_cast<const uint8_t*>(laid);
  p.x_scale = static_cast<const uint8_t*>(x_scale);
  p.begin = begin;
  p.out = out;
  p.out_scale = static_cast<uint8_t*>(out_scale);
  p.tickets = static_cast<int32_t*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                       MXFP8_EXPERT_WORKSPACE_ZEROS);
  p.flags = flags;
  e = launch_expert_product(maps, p, tile, ctas, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the experts' product");
  return MXFP8_OK;
}

mxfp8_status mxfp8_combine(const void* y, int64_t stride, int32_t slots, const float* weight,
                           const int32_t* slot, int64_t tokens, int32_t k, int32_t n,
                           const void* add, void* out, int32_t* flags, void* stream) {
  if (n < 8 || n % 8)
    return fail(MXFP8_ERR_UNSUPPORTED,
                "n must be a positive multiple of 8, got " + std::to_string(n));
  if (k < 1 || k > MXFP8_MAX_CHOICES)
    return fail(MXFP8_ERR_UNSUPPORTED, "k must be in 1.." + std::to_string(MXFP8_MAX_CHOICES) +
                                           ", got " + std::to_string(k));
  if (tokens < 0 || slots < 0)
    return fail(MXFP8_ERR_INVALID, "tokens and slots must not be negative");
  if (tokens > INT32_MAX / (n / 8))
    return fail(MXFP8_ERR_UNSUPPORTED, "tokens x n must be below 2^34");
  if (tokens == 0) return MXFP8_OK;
  if (slots > 1 && (stride < n || stride % 8))
    return fail(MXFP8_ERR_UNSUPPORTED, "the rows' stride must be at least n and a multiple of 8");
  if (slots > 0) CHECK(check_pointer("y", y, 16));
  CHECK(check_pointer("weight", weight, 4));
  CHECK(check_pointer("slot", slot, 4));
  if (add) CHECK(check_pointer("add", add, 16));
  CHECK(check_pointer("out", out, 16));
  if (flags) CHECK(check_pointer("flags", flags, 4));
  const CombineParams p{n,
                        k,
                        slots,
                        static_cast<uint32_t>(tokens * (n / 8)),
                        stride,
                        static_cast<const uint16_t*>(y),
                        weight,
                        slot,
                        static_cast<const uint16_t*>(add),
                        static_cast<uint16_t*>(out),
                        flags};
  const cudaError_t e = launch_combine(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the combination");
  return MXFP8_OK;
}

}  // extern "C"
