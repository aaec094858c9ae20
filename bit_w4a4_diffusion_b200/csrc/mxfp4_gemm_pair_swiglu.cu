// The experts' up product with SwiGLU and requantization, many rows per group,
// on CTA pairs (tcgen05 .cta_group::2): 256 rows x 128 hidden columns.
//
//   D[m, n] = sum_b Xa[m, b] Xw[n, b] sum_{k in b} a[m, k] w[n, k]    (kind::mxf4)
//   over 128 gate rows and 128 other rows of the weight;
//   h = g sigmoid(g) u, quantized to MXFP4 along the hidden columns
//
// What bounds it: mostly the operands' way from L2 to shared memory, about 84
// GB/s per SM with every SM loading; a 256-column K slice of a tile is 35 KB
// per SM (rows 16 KB, 128 weight rows 16 KB, scales 3 KB) for 256 x 256 x 256
// multiply-adds on two SMs, which keeps the tensor pipe active 63% of the time.
// After that the epilogue: without the exponential and the quotient 16 x 1024
// rows, 2048 of 4096, take 101.5 us instead of 107.7, 64 x 512 rows, 1024 of
// 2048, 61 instead of 66.  The rows are the M operand, so that a thread holds a
// row's gate and other values side by side, and whole blocks of 32 hidden
// columns.
//
// A cluster of two CTAs computes a tile: CTA r holds rows [128 r, + 128) of
// the tile, CTA 0 the gate's weight rows and CTA 1 the other factor's, the
// tensor cores exchange the weights, and each CTA accumulates its 128 rows x
// 256 columns in its own tensor memory: columns 0-255, and above them one
// 24-column scale buffer per pipeline stage, filled by the MMA warp itself
// (tcgen05.cp) right before the MMAs that read it and reused with the stage,
// so neither needs a barrier of its own.
//
// Roles (10 warps per CTA): 0-7 epilogue (tensor-memory lane quarter warp % 4,
// column half warp / 4), 8 TMA producer, 9 MMA issuer (CTA 0 only).  Barriers:
//   full[s]    CTA 0; its producer arms it with both CTAs' bytes
//   empty[s]   both CTAs; the MMA warp's commit multicasts to both
//   acc_full   both CTAs;  acc_empty  CTA 0, all 16 epilogue warps arrive
// Every mbarrier wait is bounded; both CTAs meet at the final cluster barrier.
#include "mxfp4.cuh"

namespace svdq {
namespace {

constexpr int BM = 128;                            // rows per CTA
constexpr int BN = 256;                            // weight rows per tile
constexpr int BN_HALF = BN / 2;
constexpr int BK_BYTES = 128;                      // 256 elements of K per stage
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * BK_BYTES;
constexpr int B_BYTES = BN_HALF * BK_BYTES;
constexpr int SF_BYTES = 1024;                     // 128 rows x 256 columns of scales
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 3 * SF_BYTES;   // 35 KB
static_assert(STAGE_BYTES % 1024 == 0, "stages keep the 1024-byte alignment of SWIZZLE_128B");
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9;
constexpr int NUM_THREADS = 10 * 32;
constexpr int TMEM_COLS = 512;
constexpr int SF_COLS = 24;                        // SFA 8 + SFB 16 columns per stage
constexpr int TMEM_SF0 = BN;
static_assert(TMEM_SF0 + STAGES * SF_COLS <= TMEM_COLS, "one scale buffer per stage above the accumulator");
constexpr uint16_t PAIR_MASK = 0x3;
constexpr unsigned long long kDrainLimitNs = 2000000000ull;

struct Ctl {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t acc_full;
  uint64_t acc_empty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  MxSched sched;
};
constexpr int BIAS_BYTES = EPI_WARPS * 2 * 64 * 4;  // per epilogue warp: 64 hidden columns of both factors, fp32
constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + BIAS_BYTES + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "fits the 227 KB opt-in shared memory of one CTA");

__global__ void __launch_bounds__(NUM_THREADS, 1)
    mxfp4_gemm_pair_swiglu_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfw,
                           const MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* const bias_base = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);
  Ctl* const ctl = reinterpret_cast<Ctl*>(smem + STAGES * STAGE_BYTES + BIAS_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();     // 0: leader (issues the MMAs), 1: peer
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

  // Every CTA initialises the same barrier set; only CTA 0's full[],
  // acc_empty and drain barriers are used.
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    mbar_init(smem_u32(&ctl->acc_full), 1);
    mbar_init(smem_u32(&ctl->acc_empty), 2 * EPI_WARPS);
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == PRODUCER_WARP && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_sfa);
    prefetch_tmap(&tm_sfw);
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish_pair();
  }
  // Inputs may be of the preceding kernel's making, the offsets too.
  pdl_wait();
  if (warp == 0) mx_build_sched(&ctl->sched, p.groups, p.offsets, p.rows, 2 * BM, p.dev_status);
  // Both CTAs' barriers and tensor memory exist before either is used.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  const MxSched* const sched = &ctl->sched;
  const int groups = p.groups;   // at least one: the experts' products are always grouped
  const int k_slices = (p.K + 255) / 256, k_chunks = (p.K + 127) / 128;
  const int tiles_n = (p.N + BN_HALF - 1) / BN_HALF;         // = the 128-row scale blocks of one weight matrix
  const int num_tiles = sched->pre[groups] * tiles_n;
  const WaitCtx wctx{&ctl->abort_flag, p.dev_status, p.timeout_ns};
  pdl_launch_dependents();

  if (warp == PRODUCER_WARP) {
    // -------------------------------------------------------------- producer
    int stage = 0, e = 0;
    uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
    bool ok = true;
    const uint64_t pol = policy_evict_last();   // other tiles read every operand again
    for (int tile = pair; tile < num_tiles && ok; tile += num_pairs) {
      const MxTile t = mx_decode_tile(sched, groups, tile, tiles_n, 2 * BM, e);
      const int row0 = t.row0 + (int)rank * BM;
      const int block_a = mx_first_block(sched->off[t.e], t.e) + 2 * t.mt + (int)rank;
      // The same 128 rows of the group's two matrices.
      const int row_w = (2 * t.e + (int)rank) * p.N + t.nt * BN_HALF;
      const int block_w0 = 2 * t.e * tiles_n + t.nt, block_w1 = block_w0 + tiles_n;
      for (int kb = 0; kb < k_slices; ++kb) {
        if (!mbar_wait_warp(smem_u32(&ctl->empty[stage]), phase ^ 1, wctx, kDevTimeoutProducer)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), sb = sa + A_BYTES, sf = sb + B_BYTES;
          const uint32_t local = smem_u32(&ctl->full[stage]);
          const uint32_t full = rank == 0 ? local : mapa_shared(local, 0);
          if (rank == 0) mbar_arrive_expect_tx(local, 2 * STAGE_BYTES);
          tma_load_2d_pair(sb, &tm_w, kb * BK_BYTES, row_w, full, pol);
          tma_load_2d_pair(sa, &tm_a, kb * BK_BYTES, row0, full, pol);
          // Scales: 256-byte rows, four per 128-row block and slice.
          tma_load_2d_pair(sf, &tm_sfa, 0, (block_a * k_chunks + 2 * kb) * 2, full, pol);
          tma_load_2d_pair(sf + SF_BYTES, &tm_sfw, 0, (block_w0 * k_chunks + 2 * kb) * 2, full, pol);
          tma_load_2d_pair(sf + 2 * SF_BYTES, &tm_sfw, 0, (block_w1 * k_chunks + 2 * kb) * 2, full, pol);
        }
        __syncwarp();
        issued_mask |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // CTA 0 never leaves with copies in flight into the pair's shared memory:
    // a full[] phase completes only when both CTAs' bytes landed.
    if (rank == 0) {
      volatile int never = 0;
      const WaitCtx drain_ctx{&never, p.dev_status, kDrainLimitNs};
      for (int s = 0; s < STAGES; ++s)
        if (issued_mask & (1u << s))
          mbar_wait(smem_u32(&ctl->full[s]), (issued_phase >> s) & 1, drain_ctx, kDevTimeoutDrain);
    }
  } else if (warp == MMA_WARP) {
    // -------------------------------------------------------------- MMA issuer (CTA 0)
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint32_t idesc0 = mx_idesc(2 * BM, BN, 0), idesc1 = mx_idesc(2 * BM, BN, 1);
      for (int tile = pair; tile < num_tiles && ok; tile += num_pairs) {
        // Both CTAs' epilogues have taken the previous tile's accumulator.
        if (!mbar_wait_warp(smem_u32(&ctl->acc_empty), acc_phase ^ 1, wctx, kDevTimeoutMma)) break;
        tc_fence_after();
        for (int kb = 0; kb < k_slices; ++kb) {
          if (!mbar_wait_warp(smem_u32(&ctl->full[stage]), phase, wctx, kDevTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), sb = sa + A_BYTES, ssf = sb + B_BYTES;
            const uint32_t sf = tmem + TMEM_SF0 + stage * SF_COLS;
            // 64-column steps of this slice, and the 128-column scale tiles they read.
            const int steps = min(4, (p.K - kb * 256 + 63) / 64);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (2 * j < steps) {
                tmem_cp_pair_32x128_warpx4(sf + 4 * j, mx_scale_desc(ssf + 512 * j));
                tmem_cp_pair_32x128_warpx4(sf + 8 + 8 * j, mx_scale_desc(ssf + SF_BYTES + 512 * j));
                tmem_cp_pair_32x128_warpx4(sf + 12 + 8 * j, mx_scale_desc(ssf + 2 * SF_BYTES + 512 * j));
              }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (s < steps)
                mma_mxfp4_pair(tmem, mx_operand_desc(sa + 32 * s), mx_operand_desc(sb + 32 * s),
                               s & 1 ? idesc1 : idesc0, sf + 4 * (s >> 1), sf + 8 + 8 * (s >> 1),
                               kb > 0 || s > 0 ? 1u : 0u);
            // Both CTAs may refill this stage once the MMAs reading it are done.
            tc_commit_pair_mc(smem_u32(&ctl->empty[stage]), PAIR_MASK);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_mc(smem_u32(&ctl->acc_full), PAIR_MASK);
        __syncwarp();
        acc_phase ^= 1;
      }
      // Wait for every MMA the elected lane issued before tensor memory is freed.
      if (elect_one()) tc_commit_pair(smem_u32(&ctl->drain));
      __syncwarp();
      volatile int never = 0;
      const WaitCtx drain_ctx{&never, p.dev_status, kDrainLimitNs};
      mbar_wait(smem_u32(&ctl->drain), 0, drain_ctx, kDevTimeoutDrain);
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    // A warp pulls its 32 rows x 128 columns with four loads and one wait,
    // releases the accumulator (remotely for CTA 1) and only then computes.
    const int q = warp & 3, h = warp >> 2;
    const bool fp16 = p.fp16 != 0;
    const uint32_t acc_empty_local = smem_u32(&ctl->acc_empty);
    const uint32_t acc_empty_leader = rank == 0 ? acc_empty_local : mapa_shared(acc_empty_local, 0);
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
    float* const bias_tab = bias_base + warp * 128;      // gate 64, other 64
    uint32_t acc_phase = 0;
    int e = 0;
    for (int tile = pair; tile < num_tiles; tile += num_pairs) {
      const MxTile t = mx_decode_tile(sched, groups, tile, tiles_n, 2 * BM, e);
      const int slab = (int)rank * BM + 32 * q;        // the warp's first row within the tile
      const int valid = min(32, t.rows - slab);        // its rows inside the group (may be <= 0)
      const int row0 = t.row0 + slab;
      const int nw = t.nt * BN_HALF + h * 64;          // the warp's 64 hidden columns
      if (p.bias != nullptr) {
        __syncwarp();   // the reads for the tile before are done
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = nw + 32 * (i & 1) + lane;
          bias_tab[32 * i + lane] = n < p.N ? mx_load16(p.bias + ((size_t)t.e * 2 + (i >> 1)) * p.N + n, fp16) : 0.f;
        }
        __syncwarp();
      }
      const bool got = mbar_wait(smem_u32(&ctl->acc_full), acc_phase, wctx, kDevTimeoutEpilogue);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      uint32_t r[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tmem_ld_32x32b_x32(lane_base + (uint32_t)((i >> 1) * BN_HALF + h * 64 + (i & 1) * 32), r[i]);
      }
      tmem_ld_wait(r[0]);
      reg_fence(r[1]);
      reg_fence(r[2]);
      reg_fence(r[3]);
      // The loads are complete (wait::ld) and ordered before the arrive by
      // the tcgen05 fence, which is all the MMA warp needs: CTA 1's remote
      // arrive is relaxed.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0)
          mbar_arrive(acc_empty_local);
        else
          mbar_arrive_cluster_relaxed(acc_empty_leader);
      }
      acc_phase ^= 1;
      if (valid <= 0) continue;
      // r[0..1]: gate columns nw .. + 63, r[2..3]: the other factor's.  Each
      // 32-column half is one block of the next product's K.
      const int local = t.mt * 2 * BM + slab + lane;      // row within the group
      const int block = mx_first_block(sched->off[t.e], t.e) + local / 128;
      uint8_t* const sc = p.h_scales + mx_tile_offset(block, tiles_n, t.nt) + (local & 31) * 16 +
                          (local % 128) / 32 * 4 + 2 * h;
      uint8_t* const codes = p.h_codes + (size_t)(row0 + lane) * (p.N / 2) + nw / 2;
      uint32_t bytes = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (p.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 bg = *reinterpret_cast<const float4*>(bias_tab + 32 * i + j),
                         bu = *reinterpret_cast<const float4*>(bias_tab + 64 + 32 * i + j);
            const float g4[4] = {bg.x, bg.y, bg.z, bg.w}, u4[4] = {bu.x, bu.y, bu.z, bu.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              r[i][j + x] = __float_as_uint(__fadd_rn(__uint_as_float(r[i][j + x]), g4[x]));
              r[2 + i][j + x] = __float_as_uint(__fadd_rn(__uint_as_float(r[2 + i][j + x]), u4[x]));
            }
          }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          r[i][j] = __float_as_uint(mx_swiglu(__uint_as_float(r[i][j]), __uint_as_float(r[2 + i][j])));
          top = max(top, r[i][j] & 0x7FFFFFFFu);
        }
        const uint32_t sb = mx_scale_byte(top);
        const float inv = mx_inv_scale(sb);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            v[x] = __fmul2_rn(make_float2(__uint_as_float(r[i][8 * j + 2 * x]),
                                          __uint_as_float(r[i][8 * j + 2 * x + 1])),
                              make_float2(inv, inv));
          w[j] = sb == 255u ? 0u : mx_e2m1x8(v);
        }
        const bool in_n = nw + 32 * i < p.N;              // N % 32 == 0
        bytes |= (in_n ? sb : 0u) << (8 * i);             // padding groups get byte 0
        if (in_n && lane < valid) *reinterpret_cast<uint4*>(codes + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (lane < valid) *reinterpret_cast<uint16_t*>(sc) = (uint16_t)bytes;
    }
  }

  // Both CTAs leave together: CTA 0's MMAs write CTA 1's tensor memory, and
  // CTA 1's loads count on CTA 0's barriers.
  mx_pair_meet(&ctl->abort_flag, rank);
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

}  // namespace

cudaError_t launch_mxfp4_gemm_pair_swiglu(const MxGemmParams& p, const MxGemmTmaps& t, cudaStream_t stream,
                                          bool pdl) {
  if (cudaError_t e = mx_allow_smem<mxfp4_gemm_pair_swiglu_kernel>((int)kSmemBytes)) return e;
  const long long m_tiles = mx_row_tiles(p.groups, p.rows, 2 * BM);
  return mx_launch_pairs<mxfp4_gemm_pair_swiglu_kernel, NUM_THREADS, (int)kSmemBytes>(
      m_tiles * ((p.N + BN_HALF - 1) / BN_HALF), stream, pdl, t.act, t.w, t.sfa, t.sfw, p);
}

}  // namespace svdq
