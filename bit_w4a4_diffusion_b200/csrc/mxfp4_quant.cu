// MXFP4 quantization of rows (bf16, fp16 or fp32) and its inverse.
//
//   t = max|v| over 32 along K;  scale = 2^max(floor(log2 t) - 2, -127)
//   code = E2M1(v / scale), round to nearest even, at most 6
//
// (mxfp4.cuh has the encoding and the scale layout.)  Both kernels stream:
// nothing is read twice, so HBM bounds them (2.53 bytes per element for 16-bit
// data) once there are enough rows, and the launch below that.
//
// Mapping: a CTA owns one 128-row scale block x 256 columns.  A warp takes
// the four rows r, r + 32, r + 64, r + 96 of it, whose scale bytes for four
// neighbouring groups are 16 consecutive bytes of the tiled layout: its lanes
// read 16 bytes (eight 16-bit elements) of each row, so a row's load and its
// 128-byte code store are contiguous across the warp, four lanes share a
// block's maximum by two shuffles, and a 4 x 4 byte exchange among the lanes
// of a 128-column chunk turns their scales into four aligned words.
#include "mxfp4.cuh"

namespace svdq {
namespace {

constexpr int MQ_WARPS = 8;
constexpr int MQ_THREADS = MQ_WARPS * 32;
constexpr int MQ_COLS = 256;

// The rows of scale block `block`: first row, how many (at most 128), and
// whether the block belongs to a group with sound offsets.  Every lane of the
// warp gets the same answer.
SVDQ_DEV bool find_block(int block, int rows, int groups, const int* offsets, int* dev_status, int& row0, int& count) {
  if (groups == 0) {
    row0 = block * 128;
    count = min(rows - row0, 128);
    return true;
  }
  // The last group whose first block is not behind this one.
  const int lane = threadIdx.x & 31;
  int e = -1;
  for (int base = 0; base < groups; base += 32) {
    const int i = base + lane;
    const bool le = i < groups && mx_first_block(__ldg(offsets + i), i) <= block;
    e += __popc(__ballot_sync(0xffffffffu, le));
  }
  if (e < 0) return false;
  const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
  if (lo < 0 || hi < lo || hi > rows) {
    if (lane == 0 && dev_status) atomicCAS(dev_status, 0, kDevBadIndex);
    return false;
  }
  const long long r = (long long)lo + ((long long)block - mx_first_block(lo, e)) * 128;
  if (r >= hi || r < lo) return false;
  row0 = (int)r;
  count = min(hi - row0, 128);
  return true;
}

struct Raw16 {
  uint4 w;
};
struct Raw32 {
  uint4 a, b;
};

template <int kDtype>
struct Elems;
template <>
struct Elems<kMxBf16> {
  using Raw = Raw16;
  static SVDQ_DEV Raw zero() { return {make_uint4(0, 0, 0, 0)}; }
  static SVDQ_DEV Raw load(const void* x, size_t i) {
    return {__ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i))};
  }
  static SVDQ_DEV void to_float(const Raw& r, float (&v)[8]) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Elems<kMxFp16> {
  using Raw = Raw16;
  static SVDQ_DEV Raw zero() { return {make_uint4(0, 0, 0, 0)}; }
  static SVDQ_DEV Raw load(const void* x, size_t i) { return Elems<kMxBf16>::load(x, i); }
  static SVDQ_DEV void to_float(const Raw& r, float (&v)[8]) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Elems<kMxFp32> {
  using Raw = Raw32;
  static SVDQ_DEV Raw zero() { return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
  static SVDQ_DEV Raw load(const void* x, size_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + i);
    return {__ldcs(p), __ldcs(p + 1)};
  }
  static SVDQ_DEV void to_float(const Raw& r, float (&v)[8]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
};

template <int kDtype>
__global__ void __launch_bounds__(MQ_THREADS) mxfp4_quantize_kernel(const MxQuantParams p, int k_slices) {
  using E = Elems<kDtype>;
  pdl_wait();
  // Every CTA of this grid has begun by the time a dependent kernel starts.
  pdl_launch_dependents();
  const int block = (int)(blockIdx.x / (unsigned)k_slices), slice = (int)(blockIdx.x - (unsigned)block * k_slices);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int row0, count;
  if (!find_block(block, p.rows, p.groups, p.offsets, p.dev_status, row0, count)) return;

  const int k_chunks = (p.K + 127) / 128;
  const int half = lane >> 4, l = lane & 15;            // 128-column chunk and the lane's place in it
  const int k = slice * MQ_COLS + half * 128 + 8 * l;
  const bool k_ok = k < p.K;                            // uniform over a block's four lanes
  const int chunk = slice * 2 + half;
  uint8_t* const sc = p.scales + mx_tile_offset(block, k_chunks, chunk);

  for (int r = warp; r < 32 && r < count; r += MQ_WARPS) {
    typename E::Raw raw[4];
    uint32_t lost = 0;                                  // rows whose index is out of range
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = r + 32 * i;
      raw[i] = E::zero();
      if (rr < count) {
        long long src = row0 + rr;
        if (p.row_index != nullptr) {
          src = __ldg(p.row_index + src);
          if (src < 0 || src >= p.x_rows) {
            lost |= 1u << i;
            src = -1;
          }
        }
        if (k_ok && src >= 0) raw[i] = E::load(p.x, (size_t)src * p.ldx + k);
      }
    }
    if (lost && p.dev_status) atomicCAS(p.dev_status, 0, kDevBadIndex);
    uint32_t mine = 0;                                  // byte i: the scale of row r + 32 i, this lane's block
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      E::to_float(raw[i], v);
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
      const uint32_t b = (lost >> i) & 1u ? 255u : mx_scale_byte(t);
      const float inv = mx_inv_scale(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], inv);
      const uint32_t w = b == 255u ? 0u : mx_e2m1x8(v);
      mine |= (k_ok ? b : 0u) << (8 * i);
      if (k_ok && r + 32 * i < count)
        *reinterpret_cast<uint32_t*>(p.codes + (size_t)(row0 + r + 32 * i) * (p.K / 2) + k / 2) = w;
    }
    // Lanes 0..3 of the chunk collect one row's four group bytes each.
    const uint32_t g0 = __shfl_sync(0xffffffffu, mine, half * 16), g1 = __shfl_sync(0xffffffffu, mine, half * 16 + 4),
                   g2 = __shfl_sync(0xffffffffu, mine, half * 16 + 8),
                   g3 = __shfl_sync(0xffffffffu, mine, half * 16 + 12);
    if (l < 4 && chunk < k_chunks) {
      const int s = 8 * l;
      const uint32_t w = ((g0 >> s) & 255u) | (((g1 >> s) & 255u) << 8) | (((g2 >> s) & 255u) << 16) |
                         (((g3 >> s) & 255u) << 24);
      *reinterpret_cast<uint32_t*>(sc + r * 16 + 4 * l) = w;
    }
  }
}

// Codes and scales -> values: lane l of a 128-column chunk turns the four code
// bytes at columns 8 l .. 8 l + 7 into 16 (fp32: 32) bytes.  E2M1 values times
// a power of two down to 2^-127 are exact in bf16 and fp32.
template <int kDtype>
__global__ void __launch_bounds__(MQ_THREADS) mxfp4_dequantize_kernel(const MxDequantParams p, int k_slices) {
  pdl_wait();
  pdl_launch_dependents();
  const int block = (int)(blockIdx.x / (unsigned)k_slices), slice = (int)(blockIdx.x - (unsigned)block * k_slices);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int row0, count;
  if (!find_block(block, p.rows, p.groups, p.offsets, p.dev_status, row0, count)) return;
  const int k_chunks = (p.K + 127) / 128;
  const int half = lane >> 4, l = lane & 15;
  const int k = slice * MQ_COLS + half * 128 + 8 * l;
  if (k >= p.K) return;
  const uint8_t* const sc = p.scales + mx_tile_offset(block, k_chunks, slice * 2 + half) + (l >> 2);
  for (int r = warp; r < 32 && r < count; r += MQ_WARPS) {
    uint32_t w[4];
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = b[i] = 0;
      if (r + 32 * i < count) {
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(p.codes + (size_t)(row0 + r + 32 * i) * (p.K / 2) + k / 2));
        b[i] = __ldg(sc + r * 16 + 4 * i);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r + 32 * i >= count) continue;
      // 2^(b - 127): b = 0 is the subnormal 2^-127, 255 is NaN.
      const float scale = __uint_as_float(b[i] == 255u ? 0x7FC00000u : b[i] == 0u ? 0x00400000u : b[i] << 23);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h2;   // two E2M1 codes -> two fp16 values, exact
        asm("{\n\t.reg .b8 lo, x1, x2, x3;\n\tmov.b32 {lo, x1, x2, x3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, lo;\n\t}"
            : "=r"(h2)
            : "r"(w[i] >> (8 * j)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        v[2 * j] = __fmul_rn(f.x, scale);
        v[2 * j + 1] = __fmul_rn(f.y, scale);
      }
      const size_t at = (size_t)(row0 + r + 32 * i) * p.ldo + k;
      if constexpr (kDtype == kMxFp32) {
        float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
        __stcs(out, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(out + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at),
               make_uint4(mx_pack16(v[0], v[1], false), mx_pack16(v[2], v[3], false), mx_pack16(v[4], v[5], false),
                          mx_pack16(v[6], v[7], false)));
      }
    }
  }
}

// Scale blocks of the rows: those the groups' blocks can reach.
long long row_blocks(int rows, int groups) { return groups == 0 ? ((long long)rows + 127) / 128 : rows / 128 + groups; }

template <class P, class Kernel>
cudaError_t launch_rows(const P& p, Kernel kernel, cudaStream_t stream, bool pdl) {
  const int k_slices = (p.K + MQ_COLS - 1) / MQ_COLS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(row_blocks(p.rows, p.groups) * k_slices));
  cfg.blockDim = dim3(MQ_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  set_pdl(cfg, attr, pdl);
  return cudaLaunchKernelEx(&cfg, kernel, p, k_slices);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const MxQuantParams& p, cudaStream_t stream, bool pdl) {
  switch (p.dtype) {
    case kMxBf16: return launch_rows(p, mxfp4_quantize_kernel<kMxBf16>, stream, pdl);
    case kMxFp16: return launch_rows(p, mxfp4_quantize_kernel<kMxFp16>, stream, pdl);
    default: return launch_rows(p, mxfp4_quantize_kernel<kMxFp32>, stream, pdl);
  }
}

cudaError_t launch_mxfp4_dequantize(const MxDequantParams& p, cudaStream_t stream, bool pdl) {
  if (p.dtype == kMxFp32) return launch_rows(p, mxfp4_dequantize_kernel<kMxFp32>, stream, pdl);
  return launch_rows(p, mxfp4_dequantize_kernel<kMxBf16>, stream, pdl);
}

}  // namespace svdq
