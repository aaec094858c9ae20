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

// A CTA's scale block and column slice; with parts = 4 it has one of the four
// row quads of each warp instead of all four.
struct Place {
  int block, slice, part;
};
SVDQ_DEV Place place(int k_slices, int parts) {
  const unsigned tile = blockIdx.x / (unsigned)parts, block = tile / (unsigned)k_slices;
  return {(int)block, (int)(tile - block * k_slices), (int)(blockIdx.x - tile * parts)};
}

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

template <int kDtype>
__global__ void __launch_bounds__(MQ_THREADS) mxfp4_quantize_kernel(const MxQuantParams p, int k_slices, int parts) {
  using E = MxElems<kDtype>;
  pdl_wait();
  // Every CTA of this grid has begun by the time a dependent kernel starts.
  pdl_launch_dependents();
  const Place at = place(k_slices, parts);
  const int block = at.block, slice = at.slice;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int row0, count;
  if (!find_block(block, p.rows, p.groups, p.offsets, p.dev_status, row0, count)) return;

  const int k_chunks = (p.K + 127) / 128;
  const int half = lane >> 4, l = lane & 15;            // 128-column chunk and the lane's place in it
  const int k = slice * MQ_COLS + half * 128 + 8 * l;
  const bool k_ok = k < p.K;                            // uniform over a block's four lanes
  const int chunk = slice * 2 + half;
  uint8_t* const sc = p.scales + mx_tile_offset(block, k_chunks, chunk) + 4 * l;
  const uint8_t* const x = static_cast<const uint8_t*>(p.x) + (size_t)k * E::kSize;
  const size_t pitch = (size_t)p.ldx * E::kSize;
  const bool gather = p.row_index != nullptr;

  // The warp's rows are warp + 8 t + 32 i for t, i < 4; lane 4 t + i holds
  // where row (t, i) comes from: -1 past the block's rows, -2 out of range.
  int src = -1;
  {
    const int rr = warp + MQ_WARPS * (l >> 2) + 32 * (l & 3);
    if (rr < count) {
      src = row0 + rr;
      if (gather) {
        src = __ldg(p.row_index + src);
        if (src < 0 || src >= p.x_rows) {
          src = -2;
          if (p.dev_status) atomicCAS(p.dev_status, 0, kDevBadIndex);
        }
      }
    }
  }
  auto load_quad = [&](int t, typename E::Raw (&raw)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = __shfl_sync(0xffffffffu, src, 4 * t + i);
      raw[i] = s >= 0 && k_ok ? E::load(x + (size_t)s * pitch, gather) : E::zero();
    }
  };
  auto finish_quad = [&](int t, const typename E::Raw (&raw)[4]) {
    const int r = warp + MQ_WARPS * t;
    uint32_t mine = 0;                                  // byte i: the scale of row r + 32 i, this lane's block
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = __shfl_sync(0xffffffffu, src, 4 * t + i);
      if (s == -1) continue;                            // the same in every lane
      uint32_t m = E::top(raw[i]);
      m = E::top_max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = E::top_max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t b = s == -2 ? 255u : mx_scale_byte(E::top_bits(m));
      float2 v[4];
      E::scaled(raw[i], mx_inv_scale(b), v);
      const uint32_t w = b == 255u ? 0u : mx_e2m1x8(v);
      mine |= (k_ok ? b : 0u) << (8 * i);
      if (k_ok)
        *reinterpret_cast<uint32_t*>(p.codes + (size_t)(row0 + r + 32 * i) * (p.K / 2) + k / 2) = w;
    }
    // Lanes 0..3 of the chunk collect one row's four group bytes each.
    const uint32_t g0 = __shfl_sync(0xffffffffu, mine, half * 16), g1 = __shfl_sync(0xffffffffu, mine, half * 16 + 4),
                   g2 = __shfl_sync(0xffffffffu, mine, half * 16 + 8),
                   g3 = __shfl_sync(0xffffffffu, mine, half * 16 + 12);
    if (l < 4 && chunk < k_chunks) {
      const uint32_t lo = __byte_perm(g0, g1, l | ((l + 4) << 4)), hi = __byte_perm(g2, g3, l | ((l + 4) << 4));
      *reinterpret_cast<uint32_t*>(sc + r * 16) = __byte_perm(lo, hi, 0x5410);
    }
  };
  typename E::Raw a[4], b[4];
  const int quads = min(4, (min(count, 32) - warp + MQ_WARPS - 1) / MQ_WARPS);   // those with a row
  if (parts > 1) {
    if (at.part < quads) {
      load_quad(at.part, a);
      finish_quad(at.part, a);
    }
    return;
  }
  if (quads <= 0) return;
  // The next four rows are on their way while these are worked on.
  load_quad(0, a);
  if (quads > 1) load_quad(1, b);
  finish_quad(0, a);
  if (quads > 2) load_quad(2, a);
  if (quads > 1) finish_quad(1, b);
  if (quads > 3) load_quad(3, b);
  if (quads > 2) finish_quad(2, a);
  if (quads > 3) finish_quad(3, b);
}

// Codes and scales -> values: lane l of a 128-column chunk turns the four code
// bytes at columns 8 l .. 8 l + 7 into 16 (fp32: 32) bytes.  E2M1 values times
// a power of two down to 2^-127 are exact in bf16 and fp32.
template <int kDtype>
__global__ void __launch_bounds__(MQ_THREADS) mxfp4_dequantize_kernel(const MxDequantParams p, int k_slices, int parts) {
  pdl_wait();
  pdl_launch_dependents();
  const Place at = place(k_slices, parts);
  const int block = at.block, slice = at.slice;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int row0, count;
  if (!find_block(block, p.rows, p.groups, p.offsets, p.dev_status, row0, count)) return;
  const int k_chunks = (p.K + 127) / 128;
  const int half = lane >> 4, l = lane & 15;
  const int k = slice * MQ_COLS + half * 128 + 8 * l;
  if (k >= p.K) return;
  const uint8_t* const sc = p.scales + mx_tile_offset(block, k_chunks, slice * 2 + half) + (l >> 2);
  const int r_step = MQ_WARPS * parts;
#pragma unroll 2
  for (int r = warp + MQ_WARPS * at.part; r < 32 && r < count; r += r_step) {
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

// With few tiles a warp takes one quad of rows, so that four times as many
// warps share the latency; with many it takes four and loads ahead.
constexpr long long MQ_FEW_TILES = 1024;

template <class P, class Kernel>
cudaError_t launch_rows(const P& p, Kernel kernel, cudaStream_t stream, bool pdl) {
  const int k_slices = (p.K + MQ_COLS - 1) / MQ_COLS;
  const long long tiles = row_blocks(p.rows, p.groups) * k_slices;
  const int parts = tiles < MQ_FEW_TILES ? 4 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * parts));
  cfg.blockDim = dim3(MQ_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  set_pdl(cfg, attr, pdl);
  return cudaLaunchKernelEx(&cfg, kernel, p, k_slices, parts);
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
