// C-ABI entry points of the MXFP4 operators (declared in include/svdq.h):
// argument checks, tensor maps, the choice of kernel and the launches.
// Nothing is allocated here: every buffer belongs to the caller.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <limits>

#include "svdq.h"
#include "svdq_internal.h"

using namespace svdq;

namespace {

static_assert(MXFP4_FUSED_ROWS <= kMxFusedRows && MXFP4_FUSED_GROUPED_ROWS <= kMxFusedRows, "fused kernels' limit");
static_assert(MXFP4_MAX_GROUPS == kMxMaxGroups, "header and kernels agree");
constexpr int kMaxRows = 1 << 30;   // keeps row + tile arithmetic inside 32 bits

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
long long round_up(long long a, long long b) { return (a + b - 1) / b * b; }
int elem_size(int dtype) { return dtype == kMxFp32 ? 4 : 2; }

int cuda_status(cudaError_t e, const char* what) {
  return e == cudaSuccess ? SVDQ_OK : record_error(SVDQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Scale blocks of 128 rows (groups == 0: one group of all rows).
long long scale_blocks(int groups, int rows) {
  return groups == 0 ? ((long long)rows + 127) / 128 : (long long)(rows / 128) + groups;
}
long long scale_bytes(long long blocks, int K) { return blocks * ((K + 127) / 128) * 512; }

int check_rows(int rows, int K, int groups) {
  if (rows < 0 || rows > kMaxRows)
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "rows=%d must lie in [0, %d]", rows, kMaxRows);
  if (K <= 0 || K % 32 != 0)
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "K=%d must be a positive multiple of 32", K);
  if (groups < 0 || groups > kMxMaxGroups)
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "groups=%d must lie in [0, %d]", groups, kMxMaxGroups);
  // Scale rows of 256 bytes are addressed with 32 bits, up to a block past the last.
  if (scale_bytes(scale_blocks(groups, rows) + 1, K) / 256 > std::numeric_limits<int>::max())
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "rows=%d K=%d groups=%d: too many scales", rows, K, groups);
  return SVDQ_OK;
}

int check_grid(long long ctas, const char* what) {
  if (ctas > std::numeric_limits<int>::max())
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: too many tiles for one launch", what);
  return SVDQ_OK;
}

int check_groups(int groups, const void* offsets) {
  if ((groups > 0) != (offsets != nullptr))
    return record_error(SVDQ_ERR_INVALID_ARG, "offsets must be given with groups > 0 and only then");
  if (!aligned(offsets, 4)) return record_error(SVDQ_ERR_INVALID_ARG, "offsets must be 4-byte aligned");
  return SVDQ_OK;
}

int check_matrix(const void* p, long long ld, int cols, int size, const char* what) {
  if (!p) return record_error(SVDQ_ERR_INVALID_ARG, "null pointer argument (%s)", what);
  if (!aligned(p, 16)) return record_error(SVDQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  if (ld < cols || ld * size % 16 != 0 || ld > (1ll << 40))
    return record_error(SVDQ_ERR_INVALID_ARG, "%s: row stride %lld must be at least %d and a multiple of 16 bytes",
                        what, ld, cols);
  return SVDQ_OK;
}

int check_buffer(const void* p, const char* what) {
  if (!p) return record_error(SVDQ_ERR_INVALID_ARG, "null pointer argument (%s)", what);
  if (!aligned(p, 16)) return record_error(SVDQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  return SVDQ_OK;
}

int check_product(int dtype, int rows, int N, int K, int groups, long long matrices) {
  if (dtype != kMxBf16 && dtype != kMxFp16)
    return record_error(SVDQ_ERR_INVALID_ARG, "dtype %d is not MXFP4_BF16 or MXFP4_FP16", dtype);
  if (int s = check_rows(rows, K, groups)) return s;
  if (N <= 0 || N % 8 != 0)
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "N=%d must be a positive multiple of 8", N);
  // Weight rows and their scale rows are addressed with 32 bits, up to a tile
  // (three blocks) past the last.
  const long long blocks = matrices * (((long long)N + 127) / 128) + 3;
  if (matrices * N + 384 > std::numeric_limits<int>::max() ||
      scale_bytes(blocks, K) / 256 > std::numeric_limits<int>::max())
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "%lld weights of %d x %d are too many", matrices, N, K);
  const long long m_tiles = (long long)rows / 64 + (groups == 0 ? 1 : groups);
  return check_grid(m_tiles * ((N + 127) / 128), "product");
}

struct Device {
  int sms = 0;
  int* status = nullptr;
  bool pdl = false;
};
int device(int* dev_status, Device* d) {
  if (int s = require_device(&d->sms)) return s;
  d->status = dev_status;
  if (int s = status_word(&d->status)) return s;
  d->pdl = pdl_enabled();
  return SVDQ_OK;
}

int quantize(const Device& d, int dtype, int rows, int K, const void* x, long long ldx, const int* row_index,
             int x_rows, int groups, const int* offsets, void* codes, void* scales, cudaStream_t stream) {
  MxQuantParams p{};
  p.rows = rows;
  p.K = K;
  p.dtype = dtype;
  p.x = x;
  p.ldx = ldx;
  p.row_index = row_index;
  p.x_rows = x_rows;
  p.groups = groups;
  p.offsets = offsets;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.dev_status = d.status;
  return cuda_status(launch_mxfp4_quantize(p, stream, d.pdl), "mxfp4_quantize launch");
}

// Few enough rows that the narrow kernel quantizes x itself: one launch, no
// workspace for x.  GPU time, one kernel / two, us: 4096 x 4096 6.9 / 7.3 at
// five rows, 7.0 / 7.5 at eight, 8.0 / 7.5 at twelve; 12288 x 4096 12.2 / 11.4
// at eight, 16.6 / 11.4 at twelve; and the second launch and the workspace cost
// the host 3 us.  Grouped rows count by the largest group, which
// the host does not know: up to 16 rows are rarely many of one group.
bool fuses(int groups, int rows) { return rows <= (groups == 0 ? MXFP4_FUSED_ROWS : MXFP4_FUSED_GROUPED_ROWS); }

long long narrow_m_tiles(int groups, int rows) { return mx_row_tiles(groups, rows, kMxNarrowRows); }

// SVDQ_MXFP4_GEMM_KERNEL (read at every call) forces a kernel: "narrow",
// "pair", or "pair256" / "pair384" for the pair kernel with tiles of that width.
bool forced(const char* name, size_t n) {
  const char* v = getenv("SVDQ_MXFP4_GEMM_KERNEL");
  return v && strncmp(v, name, n) == 0;
}

// Which kernel a product takes, unless one is forced.  The narrow kernel while its
// tiles fit the chip's CTA slots once, or while a group has so few rows on
// average that the weight bytes dominate.  GPU time narrow / pair, us:
//   dense, 4096 x 4096: M = 64 6.7 / 10.4, 512 10.3 / 11.2, 768 16.4 / 11.7;
//   1024 x 4096: 2048 10.4 / 11.0;  12288 x 4096: 192 11.8 / 12.3, 256 17.4 / 12.4
//   32 groups, 2048 x 2048, rows each: 96 21.0 / 22.4, 128 21.8 / 23.5, 160 27.5 / 23.9
//   SwiGLU, the same: 64 27.0 / 33.6, 96 34.7 / 33.8, 160 43.8 / 34.3
//   MLP, 32 uneven groups, 2048 x 1024: 75 rows 36.5 / 40.2, 125 46.5 / 42.9 (up product)
// The average stands for the groups, whose sizes the host does not know.  With
// most rows in one of 32 groups, 2048 x 2048, narrow / pair (* chosen), its
// share of the rows:
//   4096 rows: 30% 24.3* / 21.4, 60% 23.8* / 28.3, 90% 27.1* / 25.9;  8192 rows: 90% 41.7 / 35.8*
//   SwiGLU, 4096: 30% 41.1 / 42.5*, 60% 41.4 / 47.3*, 90% 44.8 / 47.0*;  8192: 90% 72.8 / 61.0*
bool use_pair(int groups, int rows, int N, bool swiglu, int sms) {
  if (forced("pair", 4)) return true;
  if (forced("narrow", 6)) return false;
  if (narrow_m_tiles(groups, rows) * ((N + 127) / 128) <= (long long)kMxNarrowPerSm * sms) return false;
  return rows / (groups == 0 ? 1 : groups) > (swiglu ? 96 : 128);
}

// CTAs (a cluster) that share one tile's K: as many as there are SMs for, each
// with at least four 256-column slices (SwiGLU, whose ring holds two: two), or
// as two CTAs to an SM take, each with at least eight.  GPU time, us, of 1, 2,
// 4, 8 CTAs:
//   32 tiles: 1 x 4096 x 4096 8.1, 6.3, 5.6, 5.6;  64 rows 10.4, 9.3, 8.0, 9.2
//   64 tiles: 1 x 8192 x 8192 13.6, 10.6, 9.6, 13.5;  2 experts' rows, 4096 x
//   4096 9.3, 7.3, 7.0, 11.2;  SwiGLU 15.3, 11.9, 11.1, 15.6
//   80 tiles: 77 x 5000 x 2080 8.5, 9.4;  77 x 5000 x 8192 16.6, 13.8, 15.7
//   96 tiles: 8 x 12288 x 4096 12.2, 10.6, 14.0
// With less than eight slices each, two CTAs to an SM gain nothing and leave
// an MLP's next product no room to load its weights ahead.
int choose_splits(long long tiles, int K, bool swiglu, int sms) {
  const int slices = (K + 255) / 256, least = swiglu ? 2 : 4;
  for (int s = 8; s > 1; s /= 2)
    if ((tiles * s <= sms && slices >= s * least) || (tiles * s <= (long long)kMxNarrowPerSm * sms && slices >= s * 8))
      return s;
  return 1;
}

// Parts of the pair kernel's tile: 1 (256 columns) or 2 (384), whichever takes
// fewer cycles over the rounds of the chip's CTA pairs.  A slice takes 615 or
// 809 cycles, a tile's end 1400 or 2100.  1 / 2, us: 8192^3 186.9 / 184.3;
// 4096 x 12288 x 4096 79.3 / 74.1; 16 groups of 1024, 4096 x 2048 73.1 / 70.4.
int choose_parts(int groups, int rows, int N, int K, int sms) {
  if (forced("pair256", 7)) return 1;
  if (forced("pair384", 7)) return 2;
  const double slices = (K + 255) / 256, pairs = sms / 2;
  auto cycles = [&](int cols, double slice, double end) {
    // Groups end anywhere: half a tile more for each.
    const double tiles = (groups == 0 ? (rows + 255) / 256 : rows / 256.0 + groups * 0.5) * ((N + cols - 1) / cols);
    const double rounds = groups == 0 ? std::ceil(tiles / pairs) : std::max(1.0, tiles / pairs);
    return rounds * (slices * slice + end);
  };
  return cycles(kMxPairCols<1>, 615, 1400) <= cycles(kMxPairCols<2>, 809, 2100) ? 1 : 2;
}

struct Product {
  int dtype, rows, N, K, groups;
  const int* offsets;
  const void *act_codes, *act_scales, *w_codes, *w_scales, *bias;
  void* y;
  long long ldy;
  void *h_codes, *h_scales;   // SwiGLU
  bool swiglu, weights_early;
  const void* x = nullptr;    // not null: the product quantizes x itself (act_* unused)
  long long ldx = 0;
  const int* row_index = nullptr;
  int x_rows = 0;
};

int product(const Device& d, const Product& g, cudaStream_t stream) {
  const int k_chunks = (g.K + 127) / 128;
  const int groups = g.groups == 0 ? 1 : g.groups;
  const long long matrices = (long long)groups * (g.swiglu ? 2 : 1);
  const bool pair = g.x == nullptr && use_pair(g.groups, g.rows, g.N, g.swiglu, d.sms);
  const int parts = pair && !g.swiglu ? choose_parts(g.groups, g.rows, g.N, g.K, d.sms) : 0;
  MxGemmTmaps t;
  const uint64_t sfa_rows = (uint64_t)scale_blocks(g.groups, g.rows) * k_chunks * 2;
  const uint64_t sfw_rows = (uint64_t)matrices * ((g.N + 127) / 128) * k_chunks * 2;
  bool ok = encode_tmap_2d(&t.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w_codes, g.K / 2, (uint64_t)matrices * g.N, g.K / 2,
                           128, parts == 2 ? kMxPairCols<2> / 4 : 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (g.x == nullptr) {
    ok = ok && encode_tmap_2d(&t.act, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.act_codes, g.K / 2, g.rows, g.K / 2, 128,
                              pair ? 128 : kMxNarrowBox, CU_TENSOR_MAP_SWIZZLE_128B);
    ok = ok && encode_tmap_2d(&t.sfa, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.act_scales, 256, sfa_rows, 256, 256, 4,
                              CU_TENSOR_MAP_SWIZZLE_NONE);
  } else {
    t.act = t.sfa = t.w;   // not read
  }
  ok = ok && encode_tmap_2d(&t.sfw, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w_scales, 256, sfw_rows, 256, 256, 4,
                            CU_TENSOR_MAP_SWIZZLE_NONE);
  if (pair && !g.swiglu)
    ok = ok && encode_tmap_2d(&t.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.y, g.N, g.rows, (uint64_t)g.ldy * 2, 32, 32,
                              CU_TENSOR_MAP_SWIZZLE_64B);
  else
    t.y = t.w;   // not read
  if (!ok) return record_error(SVDQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the MXFP4 product");
  MxGemmParams p{};
  p.rows = g.rows;
  p.N = g.N;
  p.K = g.K;
  p.groups = g.groups;
  p.offsets = g.offsets;
  p.bias = static_cast<const uint16_t*>(g.bias);
  p.fp16 = g.dtype == kMxFp16;
  p.y = static_cast<uint16_t*>(g.y);
  p.ldy = g.ldy;
  p.h_codes = static_cast<uint8_t*>(g.h_codes);
  p.h_scales = static_cast<uint8_t*>(g.h_scales);
  p.x = g.x;
  p.ldx = g.ldx;
  p.row_index = g.row_index;
  p.x_rows = g.x_rows;
  p.weights_early = g.weights_early && d.pdl;
  p.splits = 1;
  p.dev_status = d.status;
  p.timeout_ns = svdq_get_timeout_ns();
  if (pair && g.swiglu)
    return cuda_status(launch_mxfp4_gemm_pair_swiglu(p, t, stream, d.pdl), "mxfp4_gemm_pair_swiglu launch");
  if (pair) return cuda_status(launch_mxfp4_gemm_pair(p, t, parts, stream, d.pdl), "mxfp4_gemm_pair launch");
  const long long m_tiles = narrow_m_tiles(g.groups, g.rows);
  p.splits = choose_splits(m_tiles * ((g.N + 127) / 128), g.K, g.swiglu, d.sms);
  return cuda_status(launch_mxfp4_gemm_narrow(p, t, g.swiglu, d.sms, stream, d.pdl), "mxfp4_gemm_narrow launch");
}

// Workspace of quantized rows: codes, then scales.
long long ws_scales_offset(int rows, int K) { return round_up((long long)rows * (K / 2), 256); }
long long ws_bytes(int groups, int rows, int K) {
  return ws_scales_offset(rows, K) + round_up(scale_bytes(scale_blocks(groups, rows), K), 256);
}

int check_input(int dtype, int rows, int K, const void* x, long long ldx, const int* row_index, int x_rows) {
  if (dtype != kMxBf16 && dtype != kMxFp16 && dtype != kMxFp32)
    return record_error(SVDQ_ERR_INVALID_ARG, "dtype %d is not MXFP4_BF16, MXFP4_FP16 or MXFP4_FP32", dtype);
  if (int s = check_matrix(x, ldx, K, elem_size(dtype), "x")) return s;
  if (!aligned(row_index, 4)) return record_error(SVDQ_ERR_INVALID_ARG, "row_index must be 4-byte aligned");
  if (x_rows < 0 || (!row_index && x_rows < rows))
    return record_error(SVDQ_ERR_INVALID_ARG, "x has %d rows, %d are asked for", x_rows, rows);
  return check_grid(scale_blocks(kMxMaxGroups, rows) * ((K + 255) / 256) * kMxRowCtas, "quantize");
}

int check_workspace(const void* ws, long long have, long long need) {
  if (!ws || !aligned(ws, 16) || have < need)
    return record_error(SVDQ_ERR_INVALID_ARG, "workspace of %lld bytes (16-byte aligned) needed, %lld given", need,
                        ws ? have : 0ll);
  return SVDQ_OK;
}

// The quantized rows, then the product, on `stream`.
int linear(int dtype, int groups, int rows, int N, int K, const void* x, long long ldx, const int* row_index,
           int x_rows, const int* offsets, const void* w_codes, const void* w_scales, const void* bias, void* y,
           long long ldy, void* workspace, long long workspace_bytes, int* dev_status, void* stream) {
  if (int s = check_product(dtype, rows, N, K, groups, groups == 0 ? 1 : groups)) return s;
  if (int s = check_groups(groups, offsets)) return s;
  if (rows == 0) return SVDQ_OK;
  if (int s = check_input(dtype, rows, K, x, ldx, row_index, x_rows)) return s;
  if (int s = check_buffer(w_codes, "w_codes")) return s;
  if (int s = check_buffer(w_scales, "w_scales")) return s;
  if (!aligned(bias, 16)) return record_error(SVDQ_ERR_INVALID_ARG, "bias must be 16-byte aligned");
  if (int s = check_matrix(y, ldy, N, 2, "y")) return s;
  const bool fused = fuses(groups, rows);
  if (!fused)
    if (int s = check_workspace(workspace, workspace_bytes, ws_bytes(groups, rows, K))) return s;
  Device d;
  if (int s = device(dev_status, &d)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fused) {
    Product g{dtype, rows, N, K, groups, offsets, nullptr, nullptr, w_codes, w_scales, bias, y, ldy, nullptr, nullptr,
              false, false, x, ldx, row_index, x_rows};
    return product(d, g, st);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* scales = ws + ws_scales_offset(rows, K);
  if (int s = quantize(d, dtype, rows, K, x, ldx, row_index, x_rows, groups, offsets, ws, scales, st)) return s;
  Product g{dtype, rows, N, K, groups, offsets, ws, scales, w_codes, w_scales, bias, y, ldy, nullptr, nullptr,
            false, true};
  return product(d, g, st);
}

}  // namespace

extern "C" {

long long mxfp4_scale_bytes(int rows, int K) {
  if (rows < 0 || K <= 0 || K % 32 != 0) return -1;
  return scale_bytes(scale_blocks(0, rows), K);
}

long long mxfp4_grouped_scale_bytes(int groups, int rows, int K) {
  if (groups <= 0 || groups > kMxMaxGroups || rows < 0 || K <= 0 || K % 32 != 0) return -1;
  return scale_bytes(scale_blocks(groups, rows), K);
}

long long mxfp4_workspace_bytes(int groups, int rows, int K) {
  if (groups < 0 || groups > kMxMaxGroups || rows < 0 || K <= 0 || K % 32 != 0) return -1;
  return fuses(groups, rows) ? 0 : ws_bytes(groups, rows, K);
}

long long mxfp4_mlp_workspace_bytes(int groups, int rows, int K, int I) {
  const long long x = mxfp4_workspace_bytes(groups, rows, K);
  if (x < 0 || groups == 0 || I <= 0 || I % 32 != 0) return -1;
  return x + ws_bytes(groups, rows, I);
}

int mxfp4_quantize(int dtype, int rows, int K, const void* x, long long ldx, const int* row_index, int x_rows,
                   int groups, const int* offsets, void* codes, void* scales, int* dev_status, void* stream) {
  if (int s = check_rows(rows, K, groups)) return s;
  if (int s = check_groups(groups, offsets)) return s;
  if (rows == 0) return SVDQ_OK;
  if (int s = check_input(dtype, rows, K, x, ldx, row_index, x_rows)) return s;
  if (int s = check_buffer(codes, "codes")) return s;
  if (int s = check_buffer(scales, "scales")) return s;
  Device d;
  if (int s = device(dev_status, &d)) return s;
  return quantize(d, dtype, rows, K, x, ldx, row_index, x_rows, groups, offsets, codes, scales,
                  static_cast<cudaStream_t>(stream));
}

int mxfp4_dequantize(int dtype, int rows, int K, const void* codes, const void* scales, int groups,
                     const int* offsets, void* out, long long ldo, int* dev_status, void* stream) {
  if (int s = check_rows(rows, K, groups)) return s;
  if (int s = check_groups(groups, offsets)) return s;
  if (dtype != kMxBf16 && dtype != kMxFp32)
    return record_error(SVDQ_ERR_INVALID_ARG, "dtype %d is not MXFP4_BF16 or MXFP4_FP32", dtype);
  if (rows == 0) return SVDQ_OK;
  if (int s = check_grid(scale_blocks(kMxMaxGroups, rows) * ((K + 255) / 256) * kMxRowCtas, "dequantize")) return s;
  if (int s = check_buffer(codes, "codes")) return s;
  if (int s = check_buffer(scales, "scales")) return s;
  if (int s = check_matrix(out, ldo, K, elem_size(dtype), "out")) return s;
  Device d;
  if (int s = device(dev_status, &d)) return s;
  MxDequantParams p{rows, K, dtype, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), groups,
                    offsets, out, ldo, d.status};
  return cuda_status(launch_mxfp4_dequantize(p, static_cast<cudaStream_t>(stream), d.pdl), "mxfp4_dequantize launch");
}

int mxfp4_grouped_gemm(int dtype, int groups, int rows, int N, int K, const int* offsets, const void* act_codes,
                       const void* act_scales, const void* w_codes, const void* w_scales, const void* bias, void* y,
                       long long ldy, int* dev_status, void* stream) {
  if (int s = check_product(dtype, rows, N, K, groups, groups == 0 ? 1 : groups)) return s;
  if (int s = check_groups(groups, offsets)) return s;
  if (rows == 0) return SVDQ_OK;
  if (int s = check_buffer(act_codes, "act_codes")) return s;
  if (int s = check_buffer(act_scales, "act_scales")) return s;
  if (int s = check_buffer(w_codes, "w_codes")) return s;
  if (int s = check_buffer(w_scales, "w_scales")) return s;
  if (!aligned(bias, 16)) return record_error(SVDQ_ERR_INVALID_ARG, "bias must be 16-byte aligned");
  if (int s = check_matrix(y, ldy, N, 2, "y")) return s;
  Device d;
  if (int s = device(dev_status, &d)) return s;
  Product g{dtype, rows, N, K, groups, offsets, act_codes, act_scales, w_codes, w_scales, bias, y, ldy, nullptr,
            nullptr, false, false};
  return product(d, g, static_cast<cudaStream_t>(stream));
}

int mxfp4_gemm(int dtype, int M, int N, int K, const void* act_codes, const void* act_scales, const void* w_codes,
               const void* w_scales, const void* bias, void* y, long long ldy, int* dev_status, void* stream) {
  return mxfp4_grouped_gemm(dtype, 0, M, N, K, nullptr, act_codes, act_scales, w_codes, w_scales, bias, y, ldy,
                            dev_status, stream);
}

int mxfp4_linear(int dtype, int M, int N, int K, const void* x, long long ldx, const void* w_codes,
                 const void* w_scales, const void* bias, void* y, long long ldy, void* workspace,
                 long long workspace_bytes, int* dev_status, void* stream) {
  return linear(dtype, 0, M, N, K, x, ldx, nullptr, M, nullptr, w_codes, w_scales, bias, y, ldy, workspace,
                workspace_bytes, dev_status, stream);
}

int mxfp4_grouped_linear(int dtype, int groups, int rows, int N, int K, const void* x, long long ldx,
                         const int* row_index, int x_rows, const int* offsets, const void* w_codes,
                         const void* w_scales, const void* bias, void* y, long long ldy, void* workspace,
                         long long workspace_bytes, int* dev_status, void* stream) {
  if (groups <= 0) return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "groups=%d must be positive", groups);
  return linear(dtype, groups, rows, N, K, x, ldx, row_index, x_rows, offsets, w_codes, w_scales, bias, y, ldy,
                workspace, workspace_bytes, dev_status, stream);
}

int mxfp4_grouped_gemm_swiglu_quant(int dtype, int groups, int rows, int I, int K, const int* offsets,
                                    const void* act_codes, const void* act_scales, const void* w_codes,
                                    const void* w_scales, const void* bias, void* h_codes, void* h_scales,
                                    int* dev_status, void* stream) {
  if (groups <= 0) return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "groups=%d must be positive", groups);
  if (int s = check_product(dtype, rows, I, K, groups, 2ll * groups)) return s;
  if (int s = check_rows(rows, I, groups)) return s;   // I is the next product's K
  if (int s = check_groups(groups, offsets)) return s;
  if (rows == 0) return SVDQ_OK;
  if (int s = check_buffer(act_codes, "act_codes")) return s;
  if (int s = check_buffer(act_scales, "act_scales")) return s;
  if (int s = check_buffer(w_codes, "w_codes")) return s;
  if (int s = check_buffer(w_scales, "w_scales")) return s;
  if (!aligned(bias, 16)) return record_error(SVDQ_ERR_INVALID_ARG, "bias must be 16-byte aligned");
  if (int s = check_buffer(h_codes, "h_codes")) return s;
  if (int s = check_buffer(h_scales, "h_scales")) return s;
  Device d;
  if (int s = device(dev_status, &d)) return s;
  Product g{dtype, rows, I, K, groups, offsets, act_codes, act_scales, w_codes, w_scales, bias, nullptr, 0,
            h_codes, h_scales, true, false};
  return product(d, g, static_cast<cudaStream_t>(stream));
}

int mxfp4_grouped_mlp_swiglu(int dtype, int groups, int rows, int K, int I, const void* x, long long ldx,
                             const int* row_index, int x_rows, const int* offsets, const void* up_codes,
                             const void* up_scales, const void* up_bias, const void* down_codes,
                             const void* down_scales, const void* down_bias, void* y, long long ldy, void* workspace,
                             long long workspace_bytes, int* dev_status, void* stream) {
  if (groups <= 0) return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "groups=%d must be positive", groups);
  if (int s = check_product(dtype, rows, I, K, groups, 2ll * groups)) return s;
  if (int s = check_product(dtype, rows, K, I, groups, groups)) return s;
  if (int s = check_groups(groups, offsets)) return s;
  if (rows == 0) return SVDQ_OK;
  if (int s = check_input(dtype, rows, K, x, ldx, row_index, x_rows)) return s;
  if (int s = check_buffer(up_codes, "up_codes")) return s;
  if (int s = check_buffer(up_scales, "up_scales")) return s;
  if (int s = check_buffer(down_codes, "down_codes")) return s;
  if (int s = check_buffer(down_scales, "down_scales")) return s;
  if (!aligned(up_bias, 16) || !aligned(down_bias, 16))
    return record_error(SVDQ_ERR_INVALID_ARG, "biases must be 16-byte aligned");
  if (int s = check_matrix(y, ldy, K, 2, "y")) return s;
  if (int s = check_workspace(workspace, workspace_bytes, mxfp4_mlp_workspace_bytes(groups, rows, K, I))) return s;
  Device d;
  if (int s = device(dev_status, &d)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* xs = ws + ws_scales_offset(rows, K);
  const bool fused = fuses(groups, rows);
  uint8_t* h = ws + (fused ? 0 : ws_bytes(groups, rows, K));
  uint8_t* hs = h + ws_scales_offset(rows, I);
  Product up{dtype, rows, I, K, groups, offsets, ws, xs, up_codes, up_scales, up_bias, nullptr, 0, h, hs, true, true};
  if (fused) {
    up.x = x;
    up.ldx = ldx;
    up.row_index = row_index;
    up.x_rows = x_rows;
    up.weights_early = false;
  } else if (int s = quantize(d, dtype, rows, K, x, ldx, row_index, x_rows, groups, offsets, ws, xs, st)) {
    return s;
  }
  if (int s = product(d, up, st)) return s;
  Product down{dtype, rows, K, I, groups, offsets, h, hs, down_codes, down_scales, down_bias, y, ldy, nullptr,
               nullptr, false, true};
  return product(d, down, st);
}

}  // extern "C"
