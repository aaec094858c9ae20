// Shared pieces of the MXFP4 kernels: the scale layout, the block scale and
// element encodings, the list of row groups and the tile schedule over it.
//
// MXFP4 (OCP Microscaling Formats v1.0): E2M1 elements in blocks of 32 along
// K that share an E8M0 scale, one byte b standing for 2^(b - 127); 0xFF is
// NaN.  A block with t = max|v| gets the scale 2^max(floor(log2 t) - 2, -127)
// (section 6.3: the exponent of t less that of E2M1's largest power of two),
// and its elements v / scale round to the nearest E2M1 value, ties to even,
// at most 6 in magnitude.  A block that holds a NaN or an infinity gets 0xFF
// and zero codes, so that every product with it is NaN.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "ptx.cuh"
#include "svdq_internal.h"

namespace svdq {

// ------------------------------------------------------------------ encoding
// Scale byte of a block from the bits of max|v| (fp32, sign cleared; compared
// as integers, so that NaN and infinity win).
SVDQ_DEV uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 1 / scale, exact: the byte is at most 252, so 2^(127 - b) is normal.  Zero
// for the NaN byte, which makes every code of such a block zero.
SVDQ_DEV float mx_inv_scale(uint32_t byte) { return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23); }

// Eight fp32 -> four bytes of E2M1 codes, element 2i in bits 8i..8i+3 and
// element 2i+1 in bits 8i+4..8i+7; RNE, satfinite.
SVDQ_DEV uint32_t mx_e2m1x8(const float2 (&v)[4]) {
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(out)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return out;
}

// ------------------------------------------------------------------ elements
struct MxRaw16 {
  uint4 w;
};
struct MxRaw32 {
  uint4 a, b;
};

// Eight consecutive elements of a row: how they are loaded, their largest
// magnitude (NaN if there is one), two halves of a word for 16-bit types and
// in the end as fp32 bits, and their fp32 values times a power of two.
// Issued where it stands: not moved behind a wait to its first use.
SVDQ_DEV uint4 mx_load_now(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
SVDQ_DEV uint32_t mx_halves_max(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
template <class T2>
SVDQ_DEV uint32_t mx_max2(uint32_t a, uint32_t b) {   // NaN if either is
  const T2 m = __hmax2_nan(*reinterpret_cast<const T2*>(&a), *reinterpret_cast<const T2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <class T2>
SVDQ_DEV uint32_t mx_top8(const uint4& w) {
  const uint32_t m = 0x7FFF7FFFu;
  return mx_max2<T2>(mx_max2<T2>(w.x & m, w.y & m), mx_max2<T2>(w.z & m, w.w & m));
}

template <int kDtype>
struct MxElems;
template <>
struct MxElems<kMxBf16> {
  using Raw = MxRaw16;
  static constexpr int kSize = 2;
  static SVDQ_DEV Raw zero() { return {make_uint4(0, 0, 0, 0)}; }
  static SVDQ_DEV Raw load_now(const uint8_t* x) { return {mx_load_now(x)}; }
  static SVDQ_DEV uint32_t top(const Raw& r) { return mx_top8<__nv_bfloat162>(r.w); }
  static SVDQ_DEV uint32_t top_max(uint32_t a, uint32_t b) { return mx_max2<__nv_bfloat162>(a, b); }
  static SVDQ_DEV uint32_t top_bits(uint32_t m) { return mx_halves_max(m) << 16; }
  static SVDQ_DEV void scaled(const Raw& r, float inv, float2 (&v)[4]) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __fmul2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)),
                        make_float2(inv, inv));
  }
};
template <>
struct MxElems<kMxFp16> {
  using Raw = MxRaw16;
  static constexpr int kSize = 2;
  static SVDQ_DEV Raw zero() { return {make_uint4(0, 0, 0, 0)}; }
  static SVDQ_DEV Raw load_now(const uint8_t* x) { return {mx_load_now(x)}; }
  static SVDQ_DEV uint32_t top(const Raw& r) { return mx_top8<__half2>(r.w); }
  static SVDQ_DEV uint32_t top_max(uint32_t a, uint32_t b) { return mx_max2<__half2>(a, b); }
  static SVDQ_DEV uint32_t top_bits(uint32_t m) {
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)mx_halves_max(m))));
  }
  static SVDQ_DEV void scaled(const Raw& r, float inv, float2 (&v)[4]) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&w[i])), make_float2(inv, inv));
  }
};
template <>
struct MxElems<kMxFp32> {
  using Raw = MxRaw32;
  static constexpr int kSize = 4;
  static SVDQ_DEV Raw zero() { return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
  static SVDQ_DEV uint32_t top(const Raw& r) {
    const uint32_t m = 0x7FFFFFFFu;
    return max(max(max(r.a.x & m, r.a.y & m), max(r.a.z & m, r.a.w & m)),
               max(max(r.b.x & m, r.b.y & m), max(r.b.z & m, r.b.w & m)));
  }
  static SVDQ_DEV uint32_t top_max(uint32_t a, uint32_t b) { return max(a, b); }
  static SVDQ_DEV uint32_t top_bits(uint32_t m) { return m; }
  static SVDQ_DEV void scaled(const Raw& r, float inv, float2 (&v)[4]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __fmul2_rn(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), make_float2(inv, inv));
  }
};

// ------------------------------------------------------------------ layout
// Scales: 512-byte tiles of 128 rows x 4 blocks (128 elements of K), the
// tiles of one 128-row block next to each other: byte (row r of the block,
// group g) at (g / 4) * 512 + (r % 32) * 16 + (r / 32) * 4 + g % 4.  Rows of a
// block past the last and groups past K / 32 are padding.
SVDQ_DEV size_t mx_tile_offset(int block, int k_chunks, int chunk) {
  return ((size_t)block * k_chunks + chunk) * 512;
}

// A row's four bytes in each tile of its block.
SVDQ_DEV int mx_row_offset(int r) { return (r & 31) * 16 + (r >> 5) * 4; }

// Row groups: group e owns rows [offsets[e], offsets[e + 1]).  Its scale
// blocks begin at block offsets[e] / 128 + e: since
// floor((a + c) / 128) - floor(a / 128) + 1 >= ceil(c / 128), a group's blocks
// never reach the next group's, and no prefix sum is needed to find them.
SVDQ_DEV int mx_first_block(int offset, int e) { return (offset >> 7) + e; }

// ------------------------------------------------------------------ schedule
// Tiles of a grouped product, in shared memory: the groups' first rows and
// the running count of their row tiles.
struct MxSched {
  int off[kMxMaxGroups + 1];
  int pre[kMxMaxGroups + 1];
};

// Filled by one whole warp.  Offsets that decrease or leave [0, rows] give an
// empty schedule and a status code.  (Short code on purpose: it runs once, and
// instructions that are not in the cache yet take longer than they run.)
SVDQ_DEV void mx_build_sched(MxSched* s, int groups, const int* offsets, int rows, int tile_rows, int* dev_status) {
  const int lane = threadIdx.x & 31;
  if (groups == 0) {
    if (lane == 0) {
      s->off[0] = 0;
      s->off[1] = rows;
      s->pre[0] = 0;
      s->pre[1] = (rows + tile_rows - 1) / tile_rows;
    }
    return;
  }
#pragma unroll 4
  for (int e = lane; e <= groups; e += 32) s->off[e] = __ldg(offsets + e);
  __syncwarp();
  int run = 0;
  bool bad = false;
#pragma unroll 1
  for (int base = 0; base < groups; base += 32) {
    const int e = base + lane;
    int t = 0;
    if (e < groups) {
      const int lo = s->off[e], hi = s->off[e + 1];
      const bool wrong = lo < 0 || hi < lo || hi > rows;
      bad |= wrong;
      t = wrong ? 0 : (hi - lo + tile_rows - 1) / tile_rows;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += o;
    }
    if (e < groups) s->pre[e + 1] = run + t;
    run += __shfl_sync(0xffffffffu, t, 31);
  }
  if (lane == 0) s->pre[0] = 0;
  if (__any_sync(0xffffffffu, bad)) {
    __syncwarp();
    for (int e = lane; e <= groups; e += 32) s->pre[e] = 0;
    if (lane == 0 && dev_status) atomicCAS(dev_status, 0, kDevBadIndex);
  }
}

// One tile: row tile `mt` of group e (rows row0 .. row0 + rows - 1 of the
// matrix), column tile nt.  `tile` (less than the tile count) only grows
// between calls of one walker, which keeps the group it is in.
struct MxTile {
  int e, mt, nt, row0, rows;
};
SVDQ_DEV MxTile mx_decode_tile(const MxSched* s, int groups, int tile, int tiles_n, int tile_rows, int& e) {
  if (tile >= s->pre[e + 1] * tiles_n) {
    // The first group whose tiles end behind this one.
    int lo = e + 1, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tile >= s->pre[mid + 1] * tiles_n)
        lo = mid + 1;
      else
        hi = mid;
    }
    e = lo;
  }
  const int first = s->pre[e];
  const int local = tile - first * tiles_n, mts = s->pre[e + 1] - first;
  MxTile t;
  t.e = e;
  t.nt = mts == 1 ? local : local / mts;
  t.mt = local - t.nt * mts;
  t.row0 = s->off[e] + t.mt * tile_rows;
  t.rows = min(s->off[e + 1] - t.row0, tile_rows);
  return t;
}

// ------------------------------------------------------------------ products
// Instruction descriptor of a block-scaled product of E2M1 operands with E8M0
// scales; `step` (0 or 1) picks which two of the four scale bytes of a 32-bit
// tensor-memory word this K = 64 step uses.
SVDQ_DEV uint32_t mx_idesc(uint32_t m, uint32_t n, uint32_t step) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24) | (step << 30) | (step << 5);
}

// D[tmem] (+)= A[smem] * B[smem]^T, E2M1 x E2M1, E8M0 scales per 32 (read from
// tensor memory), fp32 accumulate.
SVDQ_DEV void mma_mxfp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa_tmem,
                        uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}
SVDQ_DEV void mma_mxfp4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa_tmem,
                             uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// Operand tiles: 128-byte rows in the 128-byte swizzle; scale tiles: rows of
// 16 bytes, eight of them 128 bytes apart.
SVDQ_DEV uint64_t mx_operand_desc(uint32_t saddr) { return smem_desc(saddr, 16, 1024, 2); }
SVDQ_DEV uint64_t mx_scale_desc(uint32_t saddr) { return smem_desc(saddr, 0, 128, 0); }

// ------------------------------------------------------------------ the end of a pair
// After a wait that gave up in either CTA of a pair, loads into the peer's
// shared memory may still be on their way, counted on a barrier that nobody
// reads any more.  Each warp tells the peer of an abort before the pair's last
// barrier, and after it both CTAs stay for as long as such loads can take.
SVDQ_DEV void mx_pair_meet(int* abort_flag, uint32_t rank) {
  if (*reinterpret_cast<volatile int*>(abort_flag) != 0)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(abort_flag), rank ^ 1u)), "r"(1)
                 : "memory");
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (*reinterpret_cast<volatile int*>(abort_flag) != 0) {
    constexpr uint64_t kStayNs = 200000;
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kStayNs) __nanosleep(1000);
  }
}

// ------------------------------------------------------------------ outputs
SVDQ_DEV float mx_load16(const uint16_t* p, bool fp16) {
  const uint16_t b = __ldg(p);
  return fp16 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
}
// Two fp32 -> two 16-bit values (a in the low half), round to nearest even.
SVDQ_DEV uint32_t mx_pack16(float a, float b, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// g sigmoid(g) u, with the exponential of -|g|, which never leaves the range
// (with exp(-g) the quotient is 0 from g = -87.3 on, where the divisor passes
// 2^126, however large u).  The exponential and the quotient are the fast
// intrinsics (relative error below 2^-20 while exp(-|g|) is normal, its last
// place of 2^-149 behind that): the value is rounded to 4 bits next.  Against
// exp(-g) alone the SwiGLU pair kernel takes 110.5 us instead of 108.7 (16 x
// 1024 rows, 2048 of 4096); no difference was found with few rows.
SVDQ_DEV float mx_swiglu(float g, float u) {
  const float t = __expf(-fabsf(g));
  const float n = g < 0.0f ? __fmul_rn(g, t) : g;
  return __fmul_rn(__fdividef(n, __fadd_rn(1.0f, t)), u);
}

}  // namespace svdq
