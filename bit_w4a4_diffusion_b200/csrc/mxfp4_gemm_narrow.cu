// MXFP4 products with few rows per group: the weight as the M operand of the
// tensor core, the rows (tokens) as its N operand.
//
//   D[n, m] = sum_b Xw[n, b] Xa[m, b] sum_{k in b} w[n, k] a[m, k]    (kind::mxf4)
//   y[m, n] = round16(D[n, m] + bias[n])
//   SwiGLU: two weights, gate and other: h = g sigmoid(g) u of their outputs,
//   quantized to MXFP4 along n for the next product
//
// What bounds it: the weight bytes.  A group with m rows does m / 0.53
// multiply-adds per weight byte, so below some 150 rows HBM is the limit and
// the kernel is a weight stream: each CTA pulls 128 weight rows x 256 columns
// (17 KB with their scales) per pipeline stage through TMA, two CTAs to an SM
// with rings of about 80 KB, which keeps more than 20 MB in flight over the
// chip, and the rows ride along as the narrow operand (N = 16 .. 64, as many
// as the tile has).
// With the weight on the M side a tile of one row costs the tensor core
// little more than its weight loads; with the rows on the M side (the pair
// kernel) it would multiply 256 rows of padding.
//
// Schedule: tiles are (group, 128 weight rows, up to 64 rows); a persistent
// CTA walks them, its producer running ahead into the next tile while the
// epilogue drains the last.  With fewer tiles than SMs a cluster of 2, 4 or 8
// CTAs shares one tile's K range and adds its partial sums through
// distributed shared memory, always in rank order.
//
// Measured (GPU time of the product): 32 groups of 32 rows, 2048 x 8192: 46.3
// us, 6.2 TB/s of weights; SwiGLU of them 86.6 us, 6.6 TB/s; 32 x 2048 x 2048
// 14.8 us, 4.8 TB/s (one CTA per SM with a ring of 200 KB took 10% more).  One
// row, 4096 x 4096: 4.9 us, of which 1 us is the preceding kernel's end, 1.8
// until the last weights are there, 0.5 the last MMAs and 1.5 the sum over the
// cluster.
//
// With a handful of rows the quantizer runs inside (kX): one more warp per
// stage reads x, a K slice at a time, and writes the codes and scale bytes of
// the row operand straight into the stage, in the layout TMA would have left.
// Every tile repeats that work, which is little for few rows, and the layer is
// one launch instead of two.
//
// Roles (6 warps): 0-3 epilogue (tensor-memory lane quarter = warp), 4 TMA
// producer, 5 MMA issuer; kX: 6 on, quantizer.  Role loops run on whole warps
// and issue from one elected lane.  Every mbarrier wait is bounded.
#include "mxfp4.cuh"

namespace svdq {
namespace {

constexpr int BW = 128;                 // weight rows per tile (MMA M)
constexpr int BK_BYTES = 128;           // 256 elements of K per stage
constexpr int EPI_WARPS = 4;
constexpr int PRODUCER_WARP = 4, MMA_WARP = 5;
constexpr int QUANT_WARP = 6;
constexpr int kNoX = -1;                // kX: x quantized beforehand, or x's dtype
constexpr int MAX_SPLITS = 8;
constexpr int H_PITCH = 36;             // words: 16-byte reads of eight rows fall into different banks
constexpr int W_BYTES = BW * BK_BYTES;  // 16 KB
constexpr int SF_BYTES = 1024;          // 128 rows x 256 columns of scales
constexpr int BOX_BYTES = kMxNarrowBox * BK_BYTES;
constexpr unsigned long long kDrainLimitNs = 2000000000ull;

// Two CTAs share an SM: one's set-up, drain and epilogue pass behind the
// other's loads, and a dependent kernel finds room before this one ends.
constexpr int TMEM_COLS = 256;
constexpr int ROWS = kMxNarrowRows;     // rows per tile (MMA N)
template <bool kGlu, int kX>
struct Cfg {
  static constexpr int kWeights = kGlu ? 2 : 1;                   // weight tiles, and accumulators, per tile
  static constexpr int kRows = kX == kNoX ? ROWS : kMxFusedRows;  // rows that a stage has room for
  static constexpr int kChunk = kRows < 32 ? kRows : 32;          // rows of one step of the epilogue
  static constexpr int kStages = kGlu ? 2 : kX == kNoX ? 3 : 4;
  static constexpr int kBufs = kGlu ? 1 : 2;                      // accumulator buffers
  static constexpr int kActBytes = kRows * BK_BYTES;
  static constexpr int kSfOff = kWeights * W_BYTES + kActBytes;   // SFW (per weight), then SFA
  static constexpr int kStageBytes = kSfOff + (kWeights + 1) * SF_BYTES;
  static constexpr int kAccRows = kRows < 32 ? 32 : kRows;        // columns of an accumulator, read 32 at a time
  static constexpr int kAccCols = kWeights * kAccRows;            // per accumulator buffer
  static constexpr int kSfCols = 8 * kWeights + 8;
  static constexpr int kTmemSf = kBufs * kAccCols;
  // Output staging: two buffers of a step's rows x 128 columns, or (SwiGLU) per
  // epilogue warp its rows x 32 hidden columns of fp32, rows 36 words apart.
  static constexpr int kStageOutBytes = kGlu ? EPI_WARPS * kChunk * H_PITCH * 4 : 2 * kChunk * BW * 2;
  static_assert(kStageBytes % 1024 == 0, "stages keep the 1024-byte alignment of SWIZZLE_128B");
  static_assert(kTmemSf + kStages * kSfCols <= TMEM_COLS, "accumulators and scale buffers fit tensor memory");
};

static_assert(kMxFusedRows == 16, "an MMA's least N; a warp's lanes hold the row index");
template <bool kGlu, int kX>
constexpr int num_threads() {           // a quantizer warp per stage
  return (QUANT_WARP + (kX == kNoX ? 0 : Cfg<kGlu, kX>::kStages)) * 32;
}

struct Ctl {
  uint64_t full[4];
  uint64_t empty[4];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int filled[4];    // kX: how often each quantizer warp filled its stage
  MxSched sched;
};

template <bool kGlu, int kX>
constexpr int smem_bytes() {
  using C = Cfg<kGlu, kX>;
  return 1024 + C::kStages * C::kStageBytes + C::kStageOutBytes + (int)sizeof(Ctl);
}
template <bool kGlu, int kX>
constexpr bool fits() {
  using C = Cfg<kGlu, kX>;
  // 228 KB per SM, 1 KB of it reserved for each CTA; partial sums reuse the ring.
  return kMxNarrowPerSm * (smem_bytes<kGlu, kX>() + 1024) <= 233472 &&
         C::kRows * C::kWeights * BW * 4 <= C::kStages * C::kStageBytes;
}
static_assert(fits<false, kNoX>() && fits<true, kNoX>() && fits<false, kMxBf16>() && fits<true, kMxBf16>(),
              "two CTAs fit an SM");

// A cluster barrier that orders nothing: the loads before it have returned,
// and the stores to y need not have (with release semantics it waits for them).
SVDQ_DEV void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
SVDQ_DEV float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <bool kGlu, int kX>
__global__ void __launch_bounds__(num_threads<kGlu, kX>(), kMxNarrowPerSm)
    mxfp4_gemm_narrow_kernel(const __grid_constant__ CUtensorMap tm_act, const __grid_constant__ CUtensorMap tm_w,
                             const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfw,
                             const MxGemmParams p) {
  using C = Cfg<kGlu, kX>;
  constexpr bool kFused = kX != kNoX;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const out_base = smem + C::kStages * C::kStageBytes;
  Ctl* const ctl = reinterpret_cast<Ctl*>(out_base + C::kStageOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), kFused ? 2 : 1);   // the producer, and a quantizer warp
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int a = 0; a < C::kBufs; ++a) {
      mbar_init(smem_u32(&ctl->acc_full[a]), 1);
      mbar_init(smem_u32(&ctl->acc_empty[a]), EPI_WARPS);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == PRODUCER_WARP && lane == 0) {
    if (!kFused) {
      prefetch_tmap(&tm_act);
      prefetch_tmap(&tm_sfa);
    }
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_sfw);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  // Scalars of the whole kernel, before the wait: its end is the start of the
  // path that a layer with few rows is made of.
  const int groups = p.groups == 0 ? 1 : p.groups;
  const int k_slices = (p.K + 255) / 256, k_chunks = (p.K + 127) / 128;
  const int tiles_n = (p.N + BW - 1) / BW;
  const int splits = p.splits, split_bits = __ffs(splits) - 1;   // a power of two
  const uint32_t rank = splits > 1 ? cluster_ctarank() : 0;
  // This CTA's part of K (whole K without splits) and its tiles.
  int kb_begin = k_slices * (int)rank >> split_bits;
  int kb_end = k_slices * ((int)rank + 1) >> split_bits;
  int t_first = (int)blockIdx.x >> split_bits, t_step = (int)gridDim.x >> split_bits;
  const MxSched* const sched = &ctl->sched;
  const WaitCtx wctx{&ctl->abort_flag, p.dev_status, p.timeout_ns};

  // Offsets are an input like the weights: with weights_early both were
  // complete before the preceding kernel began.  Without groups there are none.
  const bool sched_waits = !p.weights_early && p.groups != 0;
  if (sched_waits) pdl_wait();
  int row_index = 0;
  if (kFused && sched_waits && warp >= QUANT_WARP && p.row_index != nullptr && lane < p.rows)
    row_index = __ldg(p.row_index + lane);
  if (warp == 0) mx_build_sched(&ctl->sched, p.groups, p.offsets, p.rows, ROWS, p.dev_status);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem = ctl->tmem_base;
  int num_tiles = sched->pre[groups] * tiles_n;
  int e0 = 0;
  MxTile first = {};
  if (t_first < num_tiles) first = mx_decode_tile(sched, groups, t_first, tiles_n, ROWS, e0);
  // Computed here, not behind the wait.
  asm volatile("" : "+r"(kb_begin), "+r"(kb_end), "+r"(t_first), "+r"(t_step), "+r"(num_tiles), "+r"(tmem));
  asm volatile("" : "+r"(first.e), "+r"(first.nt), "+r"(first.mt), "+r"(first.row0), "+r"(first.rows));
  if (!p.weights_early && !sched_waits) pdl_wait();
  pdl_launch_dependents();

  if (warp == PRODUCER_WARP) {
    // -------------------------------------------------------------- producer
    int stage = 0, e = e0, issued = 0;
    uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
    bool ok = true, act_ready = !p.weights_early;
    const uint64_t pol_w = policy_evict_first(), pol_a = policy_evict_last();
    auto issue_weight = [&](int st, const MxTile& t, int kb, int boxes) {
      const uint32_t full = smem_u32(&ctl->full[st]);
      const uint32_t base = smem_u32(smem + st * C::kStageBytes);
      mbar_arrive_expect_tx(full,
                            C::kWeights * (W_BYTES + SF_BYTES) + (kFused ? 0 : boxes * BOX_BYTES + SF_BYTES));
#pragma unroll
      for (int i = 0; i < C::kWeights; ++i) {
        const int mat = t.e * C::kWeights + i;
        tma_load_2d_hint(base + i * W_BYTES, &tm_w, kb * BK_BYTES, mat * p.N + t.nt * BW, full, pol_w);
        tma_load_2d_hint(base + C::kSfOff + i * SF_BYTES, &tm_sfw, 0, ((mat * tiles_n + t.nt) * k_chunks + 2 * kb) * 2,
                         full, pol_w);
      }
    };
    auto issue_act = [&](int st, const MxTile& t, int kb, int boxes) {
      if (kFused) return;
      const uint32_t full = smem_u32(&ctl->full[st]);
      const uint32_t base = smem_u32(smem + st * C::kStageBytes);
      for (int i = 0; i < boxes; ++i)
        tma_load_2d_hint(base + C::kWeights * W_BYTES + i * BOX_BYTES, &tm_act, kb * BK_BYTES,
                         t.row0 + i * kMxNarrowBox, full, pol_a);
      const int block = (p.groups == 0 ? 0 : mx_first_block(sched->off[t.e], t.e)) + t.mt * ROWS / 128;
      tma_load_2d_hint(base + C::kSfOff + C::kWeights * SF_BYTES, &tm_sfa, 0, (block * k_chunks + 2 * kb) * 2, full,
                       pol_a);
    };
    for (int tile = t_first; tile < num_tiles && ok; tile += t_step) {
      const MxTile t = tile == t_first ? first : mx_decode_tile(sched, groups, tile, tiles_n, ROWS, e);
      const int boxes = (t.rows + kMxNarrowBox - 1) / kMxNarrowBox;
      int kb = kb_begin;
      if (!act_ready) {
        // The first stages' weight side goes out while the kernel that makes
        // the rows still runs; their row side follows once it is done.
        const int n = min(kb_end - kb_begin, C::kStages);
        if (elect_one())
          for (int i = 0; i < n; ++i) issue_weight(i, t, kb_begin + i, boxes);
        __syncwarp();
        pdl_wait();
        if (elect_one())
          for (int i = 0; i < n; ++i) issue_act(i, t, kb_begin + i, boxes);
        __syncwarp();
        for (int i = 0; i < n; ++i) {
          issued_mask |= 1u << stage;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        kb += n;
        act_ready = true;
      }
      for (; kb < kb_end; ++kb) {
        if (!mbar_wait_warp(smem_u32(&ctl->empty[stage]), phase ^ 1, wctx, kDevTimeoutProducer)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          issue_weight(stage, t, kb, boxes);
          issue_act(stage, t, kb, boxes);
        }
        __syncwarp();
        ++issued;
        issued_mask |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!act_ready) pdl_wait();
    // Never leave with copies in flight into shared memory.  A quantizer warp
    // whose wait gave up owes its stage's barrier an arrival, without which
    // the copies' phase would not end: it is made up for here, once the
    // quantizer has come to its own end.
    if constexpr (kFused) named_bar_sync(4, (1 + C::kStages) * 32);
    volatile int never = 0;
    const WaitCtx drain_ctx{&never, p.dev_status, kDrainLimitNs};
    for (int s = 0; s < C::kStages; ++s)
      if (issued_mask & (1u << s)) {
        if (kFused && lane == 0 && ctl->filled[s] < (issued + C::kStages - 1 - s) / C::kStages)
          mbar_arrive(smem_u32(&ctl->full[s]));
        __syncwarp();
        mbar_wait(smem_u32(&ctl->full[s]), (issued_phase >> s) & 1, drain_ctx, kDevTimeoutDrain);
      }
  } else if (warp == MMA_WARP) {
    // -------------------------------------------------------------- MMA issuer
    int stage = 0, e = e0, seq = 0;
    uint32_t phase = 0;
    bool ok = true;
    // Only the producer runs ahead of the preceding kernel: the others' bounded
    // waits begin behind it, so that its time does not count against them.
    if (p.weights_early) pdl_wait();
    for (int tile = t_first; tile < num_tiles && ok; tile += t_step, ++seq) {
      const MxTile t = tile == t_first ? first : mx_decode_tile(sched, groups, tile, tiles_n, ROWS, e);
      const int a = seq % C::kBufs;
      if (!mbar_wait_warp(smem_u32(&ctl->acc_empty[a]), ((seq / C::kBufs) & 1) ^ 1, wctx, kDevTimeoutMma)) break;
      tc_fence_after();
      const uint32_t n = (uint32_t)((t.rows + 15) & ~15);
      const uint32_t idesc0 = mx_idesc(BW, n, 0), idesc1 = mx_idesc(BW, n, 1);
      // The tile's rows within their 128-row scale block: 32 rows a column.
      const uint32_t sfa_off = kFused ? 0u : (uint32_t)((t.mt * ROWS % 128) / 32);
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!mbar_wait_warp(smem_u32(&ctl->full[stage]), phase, wctx, kDevTimeoutMma)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t base = smem_u32(smem + stage * C::kStageBytes);
          const uint32_t sb = base + C::kWeights * W_BYTES;
          const uint32_t sf = tmem + C::kTmemSf + stage * C::kSfCols;
          // 64-column steps of this slice, and the 128-column scale tiles they read.
          const int steps = min(4, (p.K - kb * 256 + 63) / 64);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (2 * j < steps) {
#pragma unroll
              for (int i = 0; i < C::kWeights; ++i)
                tmem_cp_32x128_warpx4(sf + 8 * i + 4 * j, mx_scale_desc(base + C::kSfOff + i * SF_BYTES + 512 * j));
              tmem_cp_32x128_warpx4(sf + 8 * C::kWeights + 4 * j,
                                    mx_scale_desc(base + C::kSfOff + C::kWeights * SF_BYTES + 512 * j));
            }
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s < steps) {
#pragma unroll
              for (int i = 0; i < C::kWeights; ++i)
                mma_mxfp4(tmem + a * C::kAccCols + i * C::kAccRows, mx_operand_desc(base + i * W_BYTES + 32 * s),
                          mx_operand_desc(sb + 32 * s), s & 1 ? idesc1 : idesc0, sf + 8 * i + 4 * (s >> 1),
                          sf + 8 * C::kWeights + 4 * (s >> 1) + sfa_off, kb > kb_begin || s > 0 ? 1u : 0u);
            }
          }
          tc_commit(smem_u32(&ctl->empty[stage]));
        }
        __syncwarp();
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(smem_u32(&ctl->acc_full[a]));
      __syncwarp();
    }
    // Wait for every MMA before tensor memory is freed.
    if (elect_one()) tc_commit(smem_u32(&ctl->drain));
    __syncwarp();
    volatile int never = 0;
    const WaitCtx drain_ctx{&never, p.dev_status, kDrainLimitNs};
    mbar_wait(smem_u32(&ctl->drain), 0, drain_ctx, kDevTimeoutDrain);
  } else if (kFused && warp >= QUANT_WARP) {
    // -------------------------------------------------------------- quantizer
    // Warp w fills stage w: lane l the eight columns 8 l .. + 7 of a slice,
    // four lanes a block.  The loads of a slice's first eight rows go out
    // together while the stage is still in use.  (One warp per stage, so that
    // each sees every phase of the one barrier that it waits on: with the
    // slices dealt out otherwise a warp could come to a barrier two phases
    // early, where its parity looks like that of the phase it wants.)
    if constexpr (kFused) {
      using E = MxElems<kX>;
      const int stage = warp - QUANT_WARP;
      uint8_t* const act = smem + stage * C::kStageBytes + C::kWeights * W_BYTES;
      uint8_t* const sf = smem + stage * C::kStageBytes + C::kSfOff + C::kWeights * SF_BYTES + (lane >> 4) * 512 +
                          ((lane >> 2) & 3);
      // Rows r .. r + N - 1 of the tile, their chains side by side.
      auto store_rows = [&](int r, uint32_t lost, const auto& raw) {
        constexpr int N = sizeof(raw) / sizeof(raw[0]);
        uint32_t m[N];
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = E::top(raw[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = E::top_max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = E::top_max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t b = (lost >> i) & 1u ? 255u : mx_scale_byte(E::top_bits(m[i]));
          float2 v[4];
          E::scaled(raw[i], mx_inv_scale(b), v);
          // 128-byte rows, 16-byte chunks XOR-ed by the row: SWIZZLE_128B.
          // Columns past K were read as zeros: codes and byte 0.
          *reinterpret_cast<uint32_t*>(act + (r + i) * 128 + (((lane >> 2) ^ ((r + i) & 7)) << 4) + (lane & 3) * 4) =
              b == 255u ? 0u : mx_e2m1x8(v);
          if ((lane & 3) == 0) sf[((r + i) & 31) * 16 + ((r + i) >> 5) * 4] = (uint8_t)b;
        }
      };
      using Raw = typename E::Raw;
      // The whole row index (at most 16 rows, one a lane), loaded at the kernel's start.
      const int index = row_index;
      int count = 0, e = e0;   // slices of all tiles so far
      int filled = 0;
      bool ok = true;
      for (int tile = t_first; tile < num_tiles && ok; tile += t_step) {
        const MxTile t = tile == t_first ? first : mx_decode_tile(sched, groups, tile, tiles_n, ROWS, e);
        for (int kb = kb_begin; kb < kb_end && ok; ++kb, ++count) {
          if (count % C::kStages != stage) continue;
          const uint32_t phase = (uint32_t)(count / C::kStages) & 1;
          const int k = kb * 256 + 8 * lane;
          const uint8_t* const x = static_cast<const uint8_t*>(p.x) + (size_t)k * E::kSize;
          for (int r0 = 0; r0 < t.rows; r0 += 8) {
            const int n = min(t.rows - r0, 8);
            Raw raw[8];
            uint32_t lost = 0;      // rows whose index is out of range
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              raw[i] = E::zero();
              if (i < n) {
                int src = t.row0 + r0 + i;
                if (p.row_index != nullptr) {
                  src = __shfl_sync(0xffffffffu, index, src);
                  if (src < 0 || src >= p.x_rows) lost |= 1u << i;
                }
                if (k < p.K && !((lost >> i) & 1u)) raw[i] = E::load_now(x + (size_t)src * p.ldx * E::kSize);
              }
            }
            if (lost && p.dev_status) atomicCAS(p.dev_status, 0, kDevBadIndex);
            if (r0 == 0 && !mbar_wait_warp(smem_u32(&ctl->empty[stage]), phase ^ 1, wctx, kDevTimeoutProducer)) {
              ok = false;
              break;
            }
            if (n == 1) {
              store_rows(r0, lost, reinterpret_cast<const Raw(&)[1]>(raw[0]));
            } else if (n == 2) {
              store_rows(r0, lost, reinterpret_cast<const Raw(&)[2]>(raw[0]));
            } else {        // up to three rows of zeros behind the tile's last are its own padding
              store_rows(r0, lost, reinterpret_cast<const Raw(&)[4]>(raw[0]));
              if (n > 4) store_rows(r0 + 4, lost >> 4, reinterpret_cast<const Raw(&)[4]>(raw[4]));
            }
          }
          if (!ok) break;
          fence_proxy_async_smem();   // the tensor core reads through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->full[stage]));
          ++filled;
        }
      }
      if (lane == 0) ctl->filled[stage] = filled;
      named_bar_sync(4, (1 + C::kStages) * 32);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    // Thread = weight row (output column); a tensor-memory column = a row of y.
    const int q = warp;
    const bool fp16 = p.fp16 != 0;
    int e = e0, seq = 0, out_seq = 0;
    if (p.weights_early) pdl_wait();
    for (int tile = t_first; tile < num_tiles; tile += t_step, ++seq) {
      const MxTile t = tile == t_first ? first : mx_decode_tile(sched, groups, tile, tiles_n, ROWS, e);
      const int a = seq % C::kBufs;
      const int n0 = t.nt * BW, n = n0 + 32 * q + lane;
      float b0 = 0.f, b1 = 0.f;
      if (p.bias != nullptr && n < p.N && splits == 1) {
        b0 = mx_load16(p.bias + (size_t)t.e * C::kWeights * p.N + n, fp16);
        if constexpr (kGlu) b1 = mx_load16(p.bias + ((size_t)t.e * 2 + 1) * p.N + n, fp16);
      }
      const bool got = mbar_wait(smem_u32(&ctl->acc_full[a]), (seq / C::kBufs) & 1, wctx, kDevTimeoutEpilogue);
      if (named_bar_any(2, EPI_WARPS * 32, !got)) break;   // decided by all four warps
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(a * C::kAccCols);
      const int chunks = (t.rows + 31) / 32;
      for (int c = 0; c < chunks; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + 32 * c, r);
        if constexpr (kGlu) {
          uint32_t r2[32];
          tmem_ld_32x32b_x32(acc + C::kAccRows + 32 * c, r2);
          tmem_ld_wait(r);
          reg_fence(r2);
          if (c == chunks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->acc_empty[a]));
          }
          if (splits > 1) {
            // Partial sums, [row][gate 128 | other 128] fp32 in the drained ring.
            float* part = reinterpret_cast<float*>(smem) + 32 * c * 2 * BW + 32 * q + lane;
#pragma unroll
            for (int j = 0; j < C::kChunk; ++j) {
              part[j * 2 * BW] = __uint_as_float(r[j]);
              part[j * 2 * BW + BW] = __uint_as_float(r2[j]);
            }
            continue;
          }
          // 32 lanes = one block of 32 hidden columns (N % 32 == 0: a warp
          // lies inside N or is padding of the last scale tile).
          const bool in_n = n0 + 32 * q < p.N;
          const int local = t.mt * ROWS + 32 * c;   // row within the group
          const int nblk = mx_first_block(sched->off[t.e], t.e) + local / 128;   // SwiGLU is always grouped
          uint8_t* const sc = p.h_scales + mx_tile_offset(nblk, tiles_n, t.nt) + (local % 128) / 32 * 4 + q;
          uint8_t* const codes = p.h_codes + (size_t)(t.row0 + 32 * c) * (p.N / 2) + (n0 + 32 * q) / 2;
          // h goes through shared memory, so that a lane then holds a row's
          // whole block: its maximum, scale and codes need no other lane.
          float* const hbuf = reinterpret_cast<float*>(out_base) + q * C::kChunk * H_PITCH;
          __syncwarp();   // the reads of the chunk before are done
#pragma unroll
          for (int j = 0; j < C::kChunk; ++j)
            hbuf[j * H_PITCH + lane] =
                mx_swiglu(__fadd_rn(__uint_as_float(r[j]), b0), __fadd_rn(__uint_as_float(r2[j]), b1));
          __syncwarp();
          if (32 * c + lane < t.rows) {
            const float4* const hrow = reinterpret_cast<const float4*>(hbuf + lane * H_PITCH);
            float4 h[8];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              h[j] = hrow[j];
              top = max(top, max(max(__float_as_uint(h[j].x) & 0x7FFFFFFFu, __float_as_uint(h[j].y) & 0x7FFFFFFFu),
                                 max(__float_as_uint(h[j].z) & 0x7FFFFFFFu, __float_as_uint(h[j].w) & 0x7FFFFFFFu)));
            }
            const uint32_t sb = mx_scale_byte(top);
            const float2 inv = make_float2(mx_inv_scale(sb), mx_inv_scale(sb));
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 v[4] = {__fmul2_rn(make_float2(h[2 * j].x, h[2 * j].y), inv),
                                   __fmul2_rn(make_float2(h[2 * j].z, h[2 * j].w), inv),
                                   __fmul2_rn(make_float2(h[2 * j + 1].x, h[2 * j + 1].y), inv),
                                   __fmul2_rn(make_float2(h[2 * j + 1].z, h[2 * j + 1].w), inv)};
              w[j] = sb == 255u ? 0u : mx_e2m1x8(v);
            }
            if (in_n) *reinterpret_cast<uint4*>(codes + (size_t)lane * (p.N / 2)) = make_uint4(w[0], w[1], w[2], w[3]);
            sc[lane * 16] = in_n ? (uint8_t)sb : (uint8_t)0;
          }
        } else {
          tmem_ld_wait(r);
          if (c == chunks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->acc_empty[a]));
          }
          if (splits > 1) {
            // Partial sums, [row][128 weight rows] fp32 in the drained ring.
            float* part = reinterpret_cast<float*>(smem) + 32 * c * BW + 32 * q + lane;
#pragma unroll
            for (int j = 0; j < C::kChunk; ++j) part[j * BW] = __uint_as_float(r[j]);
            continue;
          }
          uint8_t* const buf = out_base + (out_seq & 1) * (C::kChunk * BW * 2);
          ++out_seq;
          uint16_t* const col = reinterpret_cast<uint16_t*>(buf) + 32 * q + lane;
#pragma unroll
          for (int j = 0; j < C::kChunk; j += 2) {
            const uint32_t w = mx_pack16(__fadd_rn(__uint_as_float(r[j]), b0),
                                         __fadd_rn(__uint_as_float(r[j + 1]), b0), fp16);
            col[j * BW] = (uint16_t)w;
            col[(j + 1) * BW] = (uint16_t)(w >> 16);
          }
          // Two buffers: a thread rewrites one only after the barrier of the
          // other, which every thread reaches after its reads of the first.
          named_bar_sync(3, EPI_WARPS * 32);
#pragma unroll
          for (int i = 0; i < C::kChunk / 8; ++i) {
            const int v = threadIdx.x + 128 * i, j = v >> 4, x = v & 15;
            if (32 * c + j < t.rows && n0 + 8 * x < p.N)
              *reinterpret_cast<uint4*>(p.y + (size_t)(t.row0 + 32 * c + j) * p.ldy + n0 + 8 * x) =
                  *reinterpret_cast<const uint4*>(buf + j * (BW * 2) + x * 16);
          }
        }
      }
    }
  }

  __syncwarp();
  if (splits > 1) {
    // Every CTA of the cluster has its partial sums in place (a cluster has
    // one tile, or none); row j is added up by one warp of rank j mod splits,
    // four columns a lane.
    cluster_sync();
    if (t_first < num_tiles) {
      const MxTile t = first;
      const bool fp16 = p.fp16 != 0;
      const int n = t.nt * BW + 4 * lane;
      const bool in_n = n < p.N;          // N is a multiple of 8 (SwiGLU: 32)
      float bias[C::kWeights][4];
#pragma unroll
      for (int w = 0; w < C::kWeights; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          bias[w][i] = p.bias != nullptr && in_n
                           ? mx_load16(p.bias + ((size_t)t.e * C::kWeights + w) * p.N + n + i, fp16)
                           : 0.f;
      for (int j = (int)rank + splits * warp; j < t.rows; j += splits * (num_threads<kGlu, kX>() / 32)) {
        float v[C::kWeights][4];
#pragma unroll
        for (int w = 0; w < C::kWeights; ++w) {
          const uint32_t local = smem_u32(smem) + (uint32_t)((j * C::kWeights + w) * BW + 4 * lane) * 4;
          float4 o[MAX_SPLITS];   // all on their way before the first is added
#pragma unroll
          for (int r = 0; r < MAX_SPLITS; ++r)
            if (r < splits) o[r] = ld_cluster_f4(mapa_shared(local, (uint32_t)r));
          float4 s = o[0];
#pragma unroll
          for (int r = 1; r < MAX_SPLITS; ++r)
            if (r < splits)
              s = make_float4(__fadd_rn(s.x, o[r].x), __fadd_rn(s.y, o[r].y), __fadd_rn(s.z, o[r].z),
                              __fadd_rn(s.w, o[r].w));
          v[w][0] = __fadd_rn(s.x, bias[w][0]);
          v[w][1] = __fadd_rn(s.y, bias[w][1]);
          v[w][2] = __fadd_rn(s.z, bias[w][2]);
          v[w][3] = __fadd_rn(s.w, bias[w][3]);
        }
        if constexpr (kGlu) {
          // Eight lanes hold one block of 32 hidden columns.
          uint32_t top = 0;
          float h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[i] = mx_swiglu(v[0][i], v[1][i]);
            top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
          const uint32_t sb = mx_scale_byte(top);
          const float inv = mx_inv_scale(sb);
          const float2 v2[4] = {make_float2(__fmul_rn(h[0], inv), __fmul_rn(h[1], inv)),
                                make_float2(__fmul_rn(h[2], inv), __fmul_rn(h[3], inv)), make_float2(0.f, 0.f),
                                make_float2(0.f, 0.f)};
          const uint32_t code = sb == 255u ? 0u : mx_e2m1x8(v2);
          const int local = t.mt * ROWS + j;   // row within the group
          const int block = mx_first_block(sched->off[t.e], t.e) + local / 128;
          if (in_n)
            *reinterpret_cast<uint16_t*>(p.h_codes + (size_t)(t.row0 + j) * (p.N / 2) + n / 2) = (uint16_t)code;
          if ((lane & 7) == 0)
            p.h_scales[mx_tile_offset(block, tiles_n, t.nt) + (local & 31) * 16 + (local % 128) / 32 * 4 +
                       (lane >> 3)] = in_n ? (uint8_t)sb : (uint8_t)0;
        } else if (in_n) {
          *reinterpret_cast<uint2*>(p.y + (size_t)(t.row0 + j) * p.ldy + n) =
              make_uint2(mx_pack16(v[0][0], v[0][1], fp16), mx_pack16(v[0][2], v[0][3], fp16));
        }
      }
    }
    cluster_meet();   // no CTA leaves while its partial sums are being read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <bool kGlu, int kX>
cudaError_t launch_impl(const MxGemmParams& p, const MxGemmTmaps& t, int num_sms, cudaStream_t stream, bool pdl) {
  using C = Cfg<kGlu, kX>;
  auto kernel = mxfp4_gemm_narrow_kernel<kGlu, kX>;
  constexpr int smem = smem_bytes<kGlu, kX>();
  if (cudaError_t e = mx_allow_smem<mxfp4_gemm_narrow_kernel<kGlu, kX>>(smem)) return e;
  const long long m_tiles = mx_row_tiles(p.groups, p.rows, ROWS);
  const long long tiles = m_tiles * ((p.N + BW - 1) / BW);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.splits > 1 ? tiles * p.splits
                                             : std::min<long long>(tiles, (long long)kMxNarrowPerSm * num_sms)));
  cfg.blockDim = dim3(num_threads<kGlu, kX>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (p.splits > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)p.splits;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, t.act, t.w, t.sfa, t.sfw, p);
}

}  // namespace

cudaError_t launch_mxfp4_gemm_narrow(const MxGemmParams& p, const MxGemmTmaps& t, bool swiglu, int num_sms,
                                     cudaStream_t stream, bool pdl) {
  if (p.x == nullptr)
    return swiglu ? launch_impl<true, kNoX>(p, t, num_sms, stream, pdl)
                  : launch_impl<false, kNoX>(p, t, num_sms, stream, pdl);
  if (p.fp16)
    return swiglu ? launch_impl<true, kMxFp16>(p, t, num_sms, stream, pdl)
                  : launch_impl<false, kMxFp16>(p, t, num_sms, stream, pdl);
  return swiglu ? launch_impl<true, kMxBf16>(p, t, num_sms, stream, pdl)
                : launch_impl<false, kMxBf16>(p, t, num_sms, stream, pdl);
}

}  // namespace svdq
