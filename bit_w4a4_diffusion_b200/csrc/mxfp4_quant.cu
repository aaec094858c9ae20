// MXFP4 quantization of rows (bf16, fp16 or fp32) and its inverse.
//
//   t = max|v| over 32 along K;  scale = 2^max(floor(log2 t) - 2, -127)
//   code = E2M1(v / scale), round to nearest even, at most 6
//
// (mxfp4.cuh has the encoding and the scale layout.)  Both kernels stream:
// nothing is read twice, so HBM bounds them (2.53 bytes per element for 16-bit
// data) once there are enough rows, and the launch below that.
//
// Mapping: a warp's unit of work is four rows (a quad) by 256 columns: 32
// blocks, one per lane (lane 8 i + g: block g of row i), so that a lane finds
// its block's maximum and scale without the others.  Memory sees whole rows all the same: the quantizer
// copies the unit to shared memory with cp.async, 512 contiguous bytes of a
// row per instruction (rows may come from anywhere, so a gather costs
// nothing), and reads blocks back from there; the 16-byte chunks of a row are
// permuted so that both sides are free of bank conflicts.  All units of a
// warp are on their way before the first is worked on.  The inverse takes the same
// way back: 16 bytes of codes per lane, values through shared memory, a row's
// 512 bytes out by one bulk copy.
//
// Measured (GPU time; a device copy runs at 6.49 TB/s in the same harness):
// quantize 16384 x 8192 bf16 49.7 us, 6.83 TB/s; fp32 86.2 us, 7.05 TB/s;
// 1001 x 4096 3.1 us; 32768 rows x 2048 gathered from 8192 to 64 groups 30.3
// us, 5.6 TB/s of L2 and HBM traffic.  Dequantize 16384 x 8192 to bf16 53.6
// us, 6.33 TB/s.  With the block's maximum taken by shuffles between four lanes of 8 elements
// each, and no staging, the quantizer took 59.3 us: about 90 instructions per
// 8 elements, issue slots the limit, against about 40 here.
#include <climits>

#include "mxfp4.cuh"

namespace svdq {
namespace {

constexpr int MQ_COLS = 256;                    // columns of a unit
// Units of a warp, unless the launch spreads them.  Two against four: 4096 x
// 4096 8.7 us (9.1), 16384 x 8192 49.7 (50.2), gathered rows 30.9 (29.6).
constexpr int MQ_UNITS = 2;
// Warps per CTA: 32 KB of staging for the quantizer either way.
template <int kDtype>
constexpr int quant_warps() { return kDtype == kMxFp32 ? 4 : 8; }
template <int kDtype>
constexpr int unit_bytes() { return 4 * MQ_COLS * (kDtype == kMxFp32 ? 4 : 2); }

// The rows of quad t (0 to 31) among 128.  A whole matrix: t, t + 32, t + 64,
// t + 96, whose scales are one run of 16 bytes per chunk.  Row groups:
// neighbours, because with few rows per group a block of 128 rows of one group
// is mostly padding (1200 rows x 2080 in 32 groups: 4.0 us, against 5.7; 64 rows
// in 512 groups: 2.9 us, against 18.6; 32768 x 4096 in 8 groups: 53.2, against
// 50.9).
template <bool kGrouped>
struct Quad {
  static SVDQ_DEV int row(int t, int i) { return kGrouped ? 4 * t + i : t + 32 * i; }
  static SVDQ_DEV int count(int rows) { return kGrouped ? (rows + 3) / 4 : min(rows, 32); }   // quads with a row
};

// A warp's 128 rows and column slice, and its quads first, first + step, ....
// With `spread` a warp has one quad instead of MQ_UNITS.
struct Place {
  int block, slice, first, step;
};
template <int kWarps>
SVDQ_DEV Place place(int cta, int k_slices, int spread) {
  // CTAs of one tile (scale block x slice): 32 quads / (warps x quads each).
  constexpr unsigned kParts = 32 / (kWarps * MQ_UNITS);
  const unsigned parts = spread ? kParts * MQ_UNITS : kParts;
  const unsigned tile = cta / parts, part = cta - tile * parts;
  const unsigned block = tile / (unsigned)k_slices;
  return {(int)block, (int)(tile - block * k_slices), (int)(part * kWarps + (threadIdx.x >> 5)),
          (int)(parts * kWarps)};
}

// With groups the grid's first CTA reports offsets that decrease or leave [0,
// rows] (the others look only at those of their own rows) and does nothing
// else.  On a warp that has rows as well the check took 0.3 to 0.9 us.
SVDQ_DEV void check_offsets(int rows, int groups, const int* offsets, int* dev_status) {
  if (!dev_status) return;
  for (int e = threadIdx.x; e < groups; e += blockDim.x) {
    const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
    if (lo < 0 || hi < lo || hi > rows) atomicCAS(dev_status, 0, kDevBadIndex);
  }
}

// Where the codes and scales of one row are: its row of the matrix (-1: none,
// or of no group), the scale block and the row's place there.
struct RowPlace {
  int row, block, in_block;
};

// The place of each lane's row (lanes l and l + 8 ask for the same one).  Its
// group is the last whose first row is not behind it, found two loads deep: 32
// groups a stride apart, then those of one stride.  In groups of 128 rows and
// more on average, that of lane 0's row mostly is everyone's, so it is looked
// up first (32768 rows in 64 groups 30.3 us, against 33.3 without; 4096 rows in
// 128 groups would take 7.4, against 7.0).
SVDQ_DEV RowPlace find_row(int row, bool take, int rows, int groups, const int* offsets) {
  const int lane = threadIdx.x & 31;
  const int stride = (groups + 31) / 32;
  const int pivot = lane * stride < groups ? __ldg(offsets + lane * stride) : INT_MAX;
  int e = -1;
  bool found = false;
  if (rows >= 128 * groups) {
    const int row0 = __shfl_sync(0xffffffffu, row, 0);
    e = (__popc(__ballot_sync(0xffffffffu, pivot <= row0)) - 1) * stride;
    if (stride > 1 && e >= 0) {
      const int off = lane < stride && e + lane < groups ? __ldg(offsets + e + lane) : INT_MAX;
      e += __popc(__ballot_sync(0xffffffffu, off <= row0)) - 1;
    }
    found = __all_sync(0xffffffffu, !take || (e >= 0 && row < __ldg(offsets + e + 1)));
  }
  if (!found) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = __popc(__ballot_sync(0xffffffffu, pivot <= __shfl_sync(0xffffffffu, row, j)));
      if ((lane & 7) == j) e = (c - 1) * stride;
    }
    if (stride > 1) {
      int off[8], more = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int first = __shfl_sync(0xffffffffu, e, j), i = first + lane;
        off[j] = first >= 0 && lane < stride && i < groups ? __ldg(offsets + i) : INT_MAX;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = __popc(__ballot_sync(0xffffffffu, off[j] <= __shfl_sync(0xffffffffu, row, j)));
        if ((lane & 7) == j) more = c - 1;
      }
      e += more;
    }
  }
  if (!take || e < 0) return {-1, 0, -1};
  const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
  if (lo < 0 || row < lo || row >= hi || hi > rows) return {-1, 0, -1};
  return {row, mx_first_block(lo, e) + ((row - lo) >> 7), (row - lo) & 127};
}

// The row that this lane looks after: lane 4 t + i has row i of quad t.
template <bool kGrouped>
SVDQ_DEV RowPlace lane_row(const Place& at, int row0, int count, int rows, int groups, const int* offsets) {
  const int lane = threadIdx.x & 31;
  const int r = Quad<kGrouped>::row(at.first + at.step * ((lane >> 2) % MQ_UNITS), lane & 3);
  if (kGrouped) return find_row(row0 + r, r < count, rows, groups, offsets);
  return {r < count ? row0 + r : -1, at.block, r};
}

SVDQ_DEV void cp_async16(uint32_t dst, const void* src, bool take) {
  // Bytes not taken are zero-filled.
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
SVDQ_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SVDQ_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
SVDQ_DEV uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
SVDQ_DEV void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
SVDQ_DEV void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}

template <int kDtype, bool kGrouped>
__global__ void __launch_bounds__(quant_warps<kDtype>() * 32) mxfp4_quantize_kernel(const MxQuantParams p, int k_slices,
                                                                                   int spread) {
  using E = MxElems<kDtype>;
  constexpr int kWarps = quant_warps<kDtype>(), kUnit = unit_bytes<kDtype>();
  constexpr int kChunks = 32 * E::kSize / 16;           // 16-byte chunks of a block: 4 or 8
  extern __shared__ __align__(128) uint8_t staging[];
  if (kGrouped && blockIdx.x == 0) {
    pdl_wait();
    pdl_launch_dependents();
    check_offsets(p.rows, p.groups, p.offsets, p.dev_status);
    return;
  }
  const int cta = (int)blockIdx.x - kGrouped;
  const Place at = place<kWarps>(cta, k_slices, spread);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = at.block * 128, count = min(p.rows - row0, 128);
  const int quads_left = Quad<kGrouped>::count(count) - at.first;   // from this warp's first on
  if (quads_left <= 0) return;
  const int units = spread ? 1 : min(MQ_UNITS, (quads_left + at.step - 1) / at.step);

  const int k0 = at.slice * MQ_COLS;
  const uint32_t base = smem_u32(staging) + (uint32_t)(warp * (spread ? 1 : MQ_UNITS) * kUnit);
  const size_t pitch = (size_t)p.ldx * E::kSize;
  const uint8_t* const x = static_cast<const uint8_t*>(p.x) + (size_t)k0 * E::kSize;
  const uint32_t row_bytes = (uint32_t)min(p.K - k0, MQ_COLS) * E::kSize;
  const bool gather = p.row_index != nullptr;

  // What needs no input comes before the wait for the preceding kernel.  A
  // dependent kernel starts when every CTA is behind this point or has had
  // nothing to do, and so after the preceding kernel's end.
  pdl_wait();
  pdl_launch_dependents();
  // Lane 4 t + i holds the place of row i of the warp's quad t, and where it
  // comes from: -1 no row, or of no group, -2 out of range.
  const RowPlace mine = lane_row<kGrouped>(at, row0, count, p.rows, p.groups, p.offsets);
  int src = mine.row;
  if (gather && src >= 0) {
    src = __ldg(p.row_index + src);
    if (src < 0 || src >= p.x_rows) {
      src = -2;
      if (p.dev_status) atomicCAS(p.dev_status, 0, kDevBadIndex);
    }
  }
  // Chunk q of a row lies at chunk q ^ (what tells the blocks apart that share
  // its banks): 16-bit, blocks g and g + 2; fp32, every block.
  auto swizzle = [](int q) { return kChunks == 4 ? q ^ ((q >> 3) & 3) : q ^ ((q >> 3) & 7); };
#pragma unroll
  for (int t = 0; t < MQ_UNITS; ++t) {
    if (t < units) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = __shfl_sync(0xffffffffu, src, 4 * t + i);
        const uint8_t* const row = x + (s >= 0 ? (size_t)s * pitch : 0);
#pragma unroll
        for (int h = 0; h < kChunks / 4; ++h) {
          const int q = 32 * h + lane;
          const bool take = s >= 0 && (uint32_t)(16 * q) < row_bytes;
          cp_async16(base + t * kUnit + i * (kUnit / 4) + 16 * swizzle(q), take ? row + 16 * q : x, take);
        }
      }
    }
    cp_async_commit();
  }

  const int i = lane >> 3, g = lane & 7;                // this lane's row of a unit, and its block
  const int k_chunks = (p.K + 127) / 128;
  const int chunk = at.slice * 2 + (g >> 2);
  const bool g_ok = k0 + 32 * g < p.K;
  uint8_t* const codes = p.codes + (size_t)row0 * (p.K / 2) + k0 / 2 + 16 * g;
  auto finish = [&](int t) {
    __syncwarp();                                       // every lane's copies of the unit have landed
    const int r = Quad<kGrouped>::row(at.first + t * at.step, i);
    typename E::Raw raw[4];                             // 8 elements each
    const uint32_t row = base + t * kUnit + i * (kUnit / 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (kChunks == 4)
        raw[c] = {lds128(row + 16 * swizzle(4 * g + c))};
      else
        raw[c] = {lds128(row + 16 * swizzle(8 * g + 2 * c)), lds128(row + 16 * swizzle(8 * g + 2 * c + 1))};
    }
    const uint32_t m = E::top_max(E::top_max(E::top(raw[0]), E::top(raw[1])),
                                  E::top_max(E::top(raw[2]), E::top(raw[3])));
    uint32_t b = mx_scale_byte(E::top_bits(m));
    if (gather && __shfl_sync(0xffffffffu, src, 4 * t + i) == -2) b = 255u;
    const int block = kGrouped ? __shfl_sync(0xffffffffu, mine.block, 4 * t + i) : at.block;
    const int in_block = kGrouped ? __shfl_sync(0xffffffffu, mine.in_block, 4 * t + i) : r;
    const bool row_ok = kGrouped ? in_block >= 0 : r < count;
    const float inv = mx_inv_scale(b);
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float2 v[4];
      E::scaled(raw[c], inv, v);
      w[c] = b == 255u ? 0u : mx_e2m1x8(v);
    }
    if (g_ok && row_ok)
      *reinterpret_cast<uint4*>(codes + (size_t)r * (p.K / 2)) = make_uint4(w[0], w[1], w[2], w[3]);
    // Four lanes' bytes to one word of the scale tile (columns past K were
    // read as zeros: byte 0; rows past the last of a whole matrix too).
    uint32_t word = b << (8 * (g & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if ((g & 3) == 0 && chunk < k_chunks && (!kGrouped || row_ok))
      *reinterpret_cast<uint32_t*>(p.scales + mx_tile_offset(block, k_chunks, chunk) + mx_row_offset(in_block)) = word;
  };
  cp_async_wait<1>();
  finish(0);
  if (units > 1) {
    cp_async_wait<0>();
    finish(1);
  }
}

// Codes and scales -> values.  E2M1 values times a power of two down to 2^-127
// are exact in bf16 and fp32.
template <int kDtype, bool kGrouped>
__global__ void __launch_bounds__(8 * 32) mxfp4_dequantize_kernel(const MxDequantParams p, int k_slices, int spread) {
  constexpr int kSize = kDtype == kMxFp32 ? 4 : 2;
  constexpr int kUnit = unit_bytes<kDtype>();
  extern __shared__ __align__(128) uint8_t staging[];
  if (kGrouped && blockIdx.x == 0) {
    pdl_wait();
    pdl_launch_dependents();
    check_offsets(p.rows, p.groups, p.offsets, p.dev_status);
    return;
  }
  const int cta = (int)blockIdx.x - kGrouped;
  const Place at = place<8>(cta, k_slices, spread);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = at.block * 128, count = min(p.rows - row0, 128);
  const int quads_left = Quad<kGrouped>::count(count) - at.first;
  if (quads_left <= 0) return;
  const int units = spread ? 1 : min(MQ_UNITS, (quads_left + at.step - 1) / at.step);

  const int k0 = at.slice * MQ_COLS, k_chunks = (p.K + 127) / 128;
  const int i = lane >> 3, g = lane & 7;
  const bool g_ok = k0 + 32 * g < p.K;
  const uint8_t* const codes = p.codes + (size_t)row0 * (p.K / 2) + k0 / 2 + 16 * g;
  const int chunk = at.slice * 2 + (g >> 2);
  const uint32_t row_bytes = (uint32_t)min(p.K - k0, MQ_COLS) * kSize;
  pdl_wait();
  pdl_launch_dependents();
  const RowPlace mine = lane_row<kGrouped>(at, row0, count, p.rows, p.groups, p.offsets);
  uint4 w[MQ_UNITS];
  uint32_t b[MQ_UNITS];
#pragma unroll
  for (int t = 0; t < MQ_UNITS; ++t) {
    w[t] = make_uint4(0, 0, 0, 0);
    b[t] = 0;
    const int r = Quad<kGrouped>::row(at.first + t * at.step, i);
    const int block = kGrouped ? __shfl_sync(0xffffffffu, mine.block, 4 * t + i) : at.block;
    const int in_block = kGrouped ? __shfl_sync(0xffffffffu, mine.in_block, 4 * t + i) : r;
    if (t < units && g_ok && (kGrouped ? in_block >= 0 : r < count)) {
      w[t] = __ldcs(reinterpret_cast<const uint4*>(codes + (size_t)r * (p.K / 2)));
      b[t] = __ldg(p.scales + mx_tile_offset(block, k_chunks, chunk) + mx_row_offset(in_block) + (g & 3));
    }
  }
  // A staging buffer per unit: while one unit's rows leave, the next is made.
  const uint32_t base = smem_u32(staging) + (uint32_t)(warp * (spread ? 1 : MQ_UNITS) * kUnit);
#pragma unroll
  for (int t = 0; t < MQ_UNITS; ++t) {
    if (t >= units) break;
    const uint32_t buf = base + t * kUnit;
    // 2^(b - 127): b = 0 is the subnormal 2^-127, 255 is NaN.
    const float scale = __uint_as_float(b[t] == 255u ? 0x7FC00000u : b[t] == 0u ? 0x00400000u : b[t] << 23);
    const float2 scale2 = make_float2(scale, scale);
    const uint32_t out = buf + i * (kUnit / 4) + g * (32 * kSize);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // Word c of the lane's codes, in an order that differs between the lanes
      // that would meet in one bank.
      const int c = (s + (g >> 1)) & 3;
      const uint32_t lo = c & 1 ? w[t].y : w[t].x, hi = c & 1 ? w[t].w : w[t].z, word = c & 2 ? hi : lo;
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h2;   // two E2M1 codes -> two fp16 values, exact
        asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, x0;\n\t}"
            : "=r"(h2)
            : "r"(word >> (8 * j)));
        v[j] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h2)), scale2);
      }
      if constexpr (kDtype == kMxFp32) {
        sts128(out + 32 * c, make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                                        __float_as_uint(v[1].y)));
        sts128(out + 32 * c + 16, make_uint4(__float_as_uint(v[2].x), __float_as_uint(v[2].y),
                                             __float_as_uint(v[3].x), __float_as_uint(v[3].y)));
      } else {
        sts128(out + 16 * c, make_uint4(mx_pack16(v[0].x, v[0].y, false), mx_pack16(v[1].x, v[1].y, false),
                                        mx_pack16(v[2].x, v[2].y, false), mx_pack16(v[3].x, v[3].y, false)));
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    const int dst = __shfl_sync(0xffffffffu, mine.row, 4 * t + (lane & 3));
    if (lane < 4) {
      if (dst >= 0)
        bulk_store(static_cast<uint8_t*>(p.out) + ((size_t)dst * p.ldo + k0) * kSize, buf + lane * (kUnit / 4),
                   row_bytes);
      bulk_commit();
    }
  }
  if (lane < 4) bulk_wait<0>();
}

// With few tiles a warp takes one unit, so that twice as many warps share the
// latency (512 x 2048, 32 tiles: 2.15 us, against 2.34); with many it has all
// of its units in flight (1024 x 4096, 128 tiles: 3.0 us, against 3.8).
constexpr long long MQ_FEW_TILES = 128;

template <auto kKernel, int kWarps, int kUnit, int kBuffers, class P>
cudaError_t launch_rows(const P& p, cudaStream_t stream, bool pdl) {
  if (cudaError_t e = mx_allow_smem<kKernel>(kWarps * kBuffers * kUnit)) return e;
  const int k_slices = (p.K + MQ_COLS - 1) / MQ_COLS;
  const long long tiles = ((long long)p.rows + 127) / 128 * k_slices;
  const int spread = tiles < MQ_FEW_TILES;
  static_assert(32 / kWarps <= kMxRowCtas, "the entry points check the grid's size");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * (32 / (kWarps * MQ_UNITS)) * (spread ? MQ_UNITS : 1) + (p.groups > 0)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kWarps * (spread ? 1 : kBuffers) * kUnit;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  set_pdl(cfg, attr, pdl);
  return cudaLaunchKernelEx(&cfg, kKernel, p, k_slices, spread);
}

template <int kDtype>
cudaError_t launch_quantize(const MxQuantParams& p, cudaStream_t stream, bool pdl) {
  constexpr int kWarps = quant_warps<kDtype>();
  if (p.groups == 0)
    return launch_rows<mxfp4_quantize_kernel<kDtype, false>, kWarps, unit_bytes<kDtype>(), MQ_UNITS>(p, stream, pdl);
  return launch_rows<mxfp4_quantize_kernel<kDtype, true>, kWarps, unit_bytes<kDtype>(), MQ_UNITS>(p, stream, pdl);
}
template <int kDtype>
cudaError_t launch_dequantize(const MxDequantParams& p, cudaStream_t stream, bool pdl) {
  if (p.groups == 0)
    return launch_rows<mxfp4_dequantize_kernel<kDtype, false>, 8, unit_bytes<kDtype>(), MQ_UNITS>(p, stream, pdl);
  return launch_rows<mxfp4_dequantize_kernel<kDtype, true>, 8, unit_bytes<kDtype>(), MQ_UNITS>(p, stream, pdl);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const MxQuantParams& p, cudaStream_t stream, bool pdl) {
  switch (p.dtype) {
    case kMxBf16: return launch_quantize<kMxBf16>(p, stream, pdl);
    case kMxFp16: return launch_quantize<kMxFp16>(p, stream, pdl);
    default: return launch_quantize<kMxFp32>(p, stream, pdl);
  }
}

cudaError_t launch_mxfp4_dequantize(const MxDequantParams& p, cudaStream_t stream, bool pdl) {
  return p.dtype == kMxFp32 ? launch_dequantize<kMxFp32>(p, stream, pdl) : launch_dequantize<kMxBf16>(p, stream, pdl);
}

}  // namespace svdq
