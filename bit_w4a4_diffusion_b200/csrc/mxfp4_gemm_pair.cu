// MXFP4 products with many rows per group, on CTA pairs (tcgen05
// .cta_group::2): 256 rows x 256 or 384 weight rows per tile.
//
//   D[m, n] = sum_b Xa[m, b] Xw[n, b] sum_{k in b} a[m, k] w[n, k]    (kind::mxf4)
//   y = round16(D + bias)
//
// What bounds it: power, and the tensor pipe.  A 256-column K slice takes 615
// cycles with one part of 256 weight rows and 809 with two of 192 (512 and 768
// at the rate of the data sheet; the rest is the scale copies), and a tile
// another 1400 or 2100 while its accumulator is emptied, for which tensor
// memory has no second one.  At 8192^3 that is 295 or 280 thousand cycles, but
// the GPU then runs at about 1.5 GHz instead of 1.965: 187 and 184 us, 5.9 and
// 6.0 PFLOP/s, where cuBLAS's NVFP4 product reaches 6.1.
//
// A cluster of two CTAs computes a tile: CTA r holds rows [128 r, + 128) of
// the tile's rows and half of each part's weight rows, the tensor cores
// exchange the weight halves, and each CTA accumulates its 128 rows x all
// columns in its own tensor memory, and above them one scale buffer per
// pipeline stage, filled by the MMA warp itself (tcgen05.cp) right before the
// MMAs that read it and reused with the stage, so neither needs a barrier of
// its own.
//
// Row groups may end anywhere.  A 32-row slab that lies inside its group is
// stored by TMA; the group's last, short slab by predicated 16-byte stores,
// so that rows of the next group and rows behind the last one stay untouched.
// (With the weight as the M operand and a tile's rows as N, a group's last
// tile would cost what its rows cost; but tensor memory then holds y
// transposed, and turning it around through shared memory took more than the
// padding: 64 groups of 512 rows, 4096 x 2048, 157 us against 134.)
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
constexpr int BK_BYTES = 128;                      // 256 elements of K per stage
constexpr int A_BYTES = BM * BK_BYTES;
constexpr int SF_BYTES = 1024;                     // 128 rows x 256 columns of scales
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9;
constexpr int NUM_THREADS = 10 * 32;
constexpr int EPI_BUF_BYTES = 32 * 32 * 2;         // 32 rows x 32 columns of output
constexpr int TMEM_COLS = 512;
constexpr uint16_t PAIR_MASK = 0x3;
constexpr unsigned long long kDrainLimitNs = 2000000000ull;

template <int kParts>
struct Cfg {
  static constexpr int kPart = kMxPairCols<kParts> / kParts;               // weight rows of a part (MMA N)
  static constexpr int kCols = kParts * kPart;
  static constexpr int kPartBytes = kPart / 2 * BK_BYTES;                  // a CTA's half of a part
  static constexpr int kSfOff = A_BYTES + kParts * kPartBytes;             // SFA, then the tile's SFB blocks
  static constexpr int kBlocks = kCols / 128;
  static constexpr int kStageBytes = kSfOff + (1 + kBlocks) * SF_BYTES;    // 35 or 44 KB
  static constexpr int kStages = kParts == 1 ? 5 : 4;
  static constexpr int kWarpCols = kCols / 2;                              // accumulator columns per epilogue warp
  static constexpr int kBiasBytes = EPI_WARPS * kWarpCols * 4;
  static constexpr int kEpiBytes = EPI_WARPS * 2 * EPI_BUF_BYTES + kBiasBytes;
  static constexpr int kSfCols = 8 + 8 * kBlocks;                          // per stage
  static constexpr int kTmemSf = kCols;
  static_assert(kStageBytes % 1024 == 0 && kPartBytes % 1024 == 0, "SWIZZLE_128B tiles stay 1024-byte aligned");
  static_assert(kTmemSf + kStages * kSfCols <= TMEM_COLS, "one scale buffer per stage above the accumulator");
};

template <int kParts>
struct Ctl {
  uint64_t full[Cfg<kParts>::kStages];
  uint64_t empty[Cfg<kParts>::kStages];
  uint64_t acc_full;
  uint64_t acc_empty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  MxSched sched;
};
template <int kParts>
constexpr int smem_bytes() {
  return 1024 + Cfg<kParts>::kStages * Cfg<kParts>::kStageBytes + Cfg<kParts>::kEpiBytes + (int)sizeof(Ctl<kParts>);
}
static_assert(smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448, "fits the shared memory of one CTA");

template <int kParts>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    mxfp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfw,
                           const __grid_constant__ CUtensorMap tm_y, const MxGemmParams p) {
  using C = Cfg<kParts>;
  constexpr int STAGES = C::kStages, STAGE_BYTES = C::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const epi_base = smem + STAGES * STAGE_BYTES;
  Ctl<kParts>* const ctl = reinterpret_cast<Ctl<kParts>*>(epi_base + C::kEpiBytes);
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
    prefetch_tmap(&tm_y);
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish_pair();
  }
  // Inputs may be of the preceding kernel's making, the offsets too; without
  // groups all that comes before the loads goes before the wait.
  if (p.groups != 0) pdl_wait();
  if (warp == 0) mx_build_sched(&ctl->sched, p.groups, p.offsets, p.rows, 2 * BM, p.dev_status);
  // Both CTAs' barriers and tensor memory exist before either is used.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  const MxSched* const sched = &ctl->sched;
  const int groups = p.groups == 0 ? 1 : p.groups;
  const int k_slices = (p.K + 255) / 256, k_chunks = (p.K + 127) / 128;
  const int tiles_n = (p.N + C::kCols - 1) / C::kCols;
  const int blocks_n = (p.N + 127) / 128;                    // 128-row scale blocks of one weight matrix
  const int num_tiles = sched->pre[groups] * tiles_n;
  const WaitCtx wctx{&ctl->abort_flag, p.dev_status, p.timeout_ns};
  if (p.groups == 0) pdl_wait();
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
      const int block_a = (p.groups == 0 ? 0 : mx_first_block(sched->off[t.e], t.e)) + 2 * t.mt + (int)rank;
      const int row_w = t.e * p.N + t.nt * C::kCols + (int)rank * (C::kPart / 2);
      const int block_w = t.e * blocks_n + t.nt * C::kBlocks;
      for (int kb = 0; kb < k_slices; ++kb) {
        if (!mbar_wait_warp(smem_u32(&ctl->empty[stage]), phase ^ 1, wctx, kDevTimeoutProducer)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), sb = sa + A_BYTES, sf = sa + C::kSfOff;
          const uint32_t local = smem_u32(&ctl->full[stage]);
          const uint32_t full = rank == 0 ? local : mapa_shared(local, 0);
          if (rank == 0) mbar_arrive_expect_tx(local, 2 * STAGE_BYTES);
#pragma unroll
          for (int i = 0; i < kParts; ++i)
            tma_load_2d_pair(sb + i * C::kPartBytes, &tm_w, kb * BK_BYTES, row_w + i * C::kPart, full, pol);
          tma_load_2d_pair(sa, &tm_a, kb * BK_BYTES, row0, full, pol);
          // Scales: 256-byte rows, four per 128-row block and slice.
          tma_load_2d_pair(sf, &tm_sfa, 0, (block_a * k_chunks + 2 * kb) * 2, full, pol);
#pragma unroll
          for (int i = 0; i < C::kBlocks; ++i)
            tma_load_2d_pair(sf + (1 + i) * SF_BYTES, &tm_sfw, 0, ((block_w + i) * k_chunks + 2 * kb) * 2, full, pol);
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
      const uint32_t idesc0 = mx_idesc(2 * BM, C::kPart, 0), idesc1 = mx_idesc(2 * BM, C::kPart, 1);
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
            const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), ssf = sa + C::kSfOff;
            const uint32_t sf = tmem + C::kTmemSf + stage * C::kSfCols;
            // 64-column steps of this slice, and the 128-column scale tiles they read.
            const int steps = min(4, (p.K - kb * 256 + 63) / 64);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (2 * j < steps) {
                tmem_cp_pair_32x128_warpx4(sf + 4 * j, mx_scale_desc(ssf + 512 * j));
#pragma unroll
                for (int i = 0; i < C::kBlocks; ++i)
                  tmem_cp_pair_32x128_warpx4(sf + 8 + 4 * C::kBlocks * j + 4 * i,
                                             mx_scale_desc(ssf + (1 + i) * SF_BYTES + 512 * j));
              }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int i = 0; i < kParts; ++i)
                if (s < steps)
                  mma_mxfp4_pair(tmem + i * C::kPart, mx_operand_desc(sa + 32 * s),
                                 mx_operand_desc(sa + A_BYTES + i * C::kPartBytes + 32 * s), s & 1 ? idesc1 : idesc0,
                                 sf + 4 * (s >> 1), sf + 8 + 4 * C::kBlocks * (s >> 1) + i * (C::kPart / 32),
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
    // A warp adds the bias and rounds to 16 bits as it loads its 32 rows x
    // half of the columns, releases the accumulator (remotely for CTA 1) and
    // only then stores.
    const int q = warp & 3, h = warp >> 2;
    const bool fp16 = p.fp16 != 0;
    uint8_t* const buf0 = epi_base + warp * 2 * EPI_BUF_BYTES;
    float* const bias_tab = reinterpret_cast<float*>(epi_base + EPI_WARPS * 2 * EPI_BUF_BYTES) + warp * C::kWarpCols;
    const uint32_t acc_empty_local = smem_u32(&ctl->acc_empty);
    const uint32_t acc_empty_leader = rank == 0 ? acc_empty_local : mapa_shared(acc_empty_local, 0);
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(h * C::kWarpCols);
    uint32_t acc_phase = 0;
    int store_seq = 0, e = 0;
    for (int tile = pair; tile < num_tiles; tile += num_pairs) {
      const MxTile t = mx_decode_tile(sched, groups, tile, tiles_n, 2 * BM, e);
      const int slab = (int)rank * BM + 32 * q;        // the warp's first row within the tile
      const int valid = min(32, t.rows - slab);        // its rows inside the group (may be <= 0)
      const int row0 = t.row0 + slab;
      const int nw = t.nt * C::kCols + h * C::kWarpCols;
      if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < C::kWarpCols / 32; ++i) {
          const int n = nw + 32 * i + lane;
          bias_tab[32 * i + lane] = n < p.N ? mx_load16(p.bias + (size_t)t.e * p.N + n, fp16) : 0.f;
        }
        __syncwarp();
      }
      const bool got = mbar_wait(smem_u32(&ctl->acc_full), acc_phase, wctx, kDevTimeoutEpilogue);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      uint32_t out[C::kWarpCols / 32][16];
#pragma unroll
      for (int i = 0; i < C::kWarpCols / 32; ++i) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + 32 * i, r);
        tmem_ld_wait(r);
        if (p.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 b = reinterpret_cast<const float4*>(bias_tab + 32 * i)[j];
            const float2 lo = __fadd2_rn(make_float2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])),
                                         make_float2(b.x, b.y));
            const float2 hi = __fadd2_rn(make_float2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                                         make_float2(b.z, b.w));
            out[i][2 * j] = mx_pack16(lo.x, lo.y, fp16);
            out[i][2 * j + 1] = mx_pack16(hi.x, hi.y, fp16);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            out[i][j] = mx_pack16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), fp16);
        }
      }
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
#pragma unroll
      for (int i = 0; i < C::kWarpCols / 32; ++i) {
        const int ncol = nw + 32 * i;
        if (valid == 32) {
          uint8_t* const buf = buf0 + (store_seq & 1) * EPI_BUF_BYTES;
          if (lane == 0) bulk_wait_read<1>();   // the store two pieces ago has read this buffer
          __syncwarp();
          uint8_t* const row = buf + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int pj = j ^ ((lane >> 1) & 3);  // 64-byte swizzle
            *reinterpret_cast<uint4*>(row + pj * 16) =
                make_uint4(out[i][4 * j], out[i][4 * j + 1], out[i][4 * j + 2], out[i][4 * j + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ncol < p.N) tma_store_2d(&tm_y, ncol, row0, smem_u32(buf));
          if (lane == 0) bulk_commit();
          ++store_seq;
        } else if (lane < valid) {
          uint16_t* const y = p.y + (size_t)(row0 + lane) * p.ldy + ncol;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (ncol + 8 * j < p.N)
              *reinterpret_cast<uint4*>(y + 8 * j) =
                  make_uint4(out[i][4 * j], out[i][4 * j + 1], out[i][4 * j + 2], out[i][4 * j + 3]);
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
  }

  // Both CTAs leave together: CTA 0's MMAs write CTA 1's tensor memory, and
  // CTA 1's loads count on CTA 0's barriers.
  mx_pair_meet(&ctl->abort_flag, rank);
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

template <int kParts>
cudaError_t launch_impl(const MxGemmParams& p, const MxGemmTmaps& t, cudaStream_t stream, bool pdl) {
  constexpr int kSmem = smem_bytes<kParts>(), kCols = Cfg<kParts>::kCols;
  if (cudaError_t e = mx_allow_smem<mxfp4_gemm_pair_kernel<kParts>>(kSmem)) return e;
  const long long m_tiles = mx_row_tiles(p.groups, p.rows, 2 * BM);
  return mx_launch_pairs<mxfp4_gemm_pair_kernel<kParts>, NUM_THREADS, kSmem>(
      m_tiles * ((p.N + kCols - 1) / kCols), stream, pdl, t.act, t.w, t.sfa, t.sfw, t.y, p);
}

}  // namespace

cudaError_t launch_mxfp4_gemm_pair(const MxGemmParams& p, const MxGemmTmaps& t, int parts, cudaStream_t stream,
                                   bool pdl) {
  return parts == 2 ? launch_impl<2>(p, t, stream, pdl) : launch_impl<1>(p, t, stream, pdl);
}

}  // namespace svdq
