// project.cu -- FP4 projections with more work in the tile than a product:
// tiles of 256 rows on CTA pairs (rows.cu has the form for few rows).
//
//   GATED    H[m, j] = act(G[m, j]) U[m, j],  G | U = X W^T with W = [Wg; Wu]
//            one [2F, C] operand: a tile holds 128 columns of G and the same
//            128 columns of U, so the activation and the product happen in the
//            registers of the thread that reads the accumulators and H (and,
//            for training, G | U) is all that is written.
//   ADAPTER  Y = X W^T + scale_i (X A_i^T) B_i^T: after the FP4 K steps of a
//            tile, the low-rank product runs as BF16 K steps into the same
//            accumulator.  Its first operand, V = scale_i X A_i^T divided by
//            the FP4 product's decode scale, comes as one 256-row slab for
//            each adapter that a row tile has rows of, zero in the other rows
//            (operands.cu builds them), so a tile whose rows use several adapters
//            adds K steps for each: one for every 32 ranks, whose 64 columns of
//            the slab are V's two BF16 terms, both by the same 32 ranks of B.
//            Where V over the decode scale leaves FP32's range, a tile has no
//            such steps: its epilogue adds V's products in FP32 (slow, and rare:
//            scales whose product is next to nothing, adapters out of all
//            proportion to W).
//
// The pipeline: a cluster of two CTAs computes a 256 x 256 accumulator tile,
// persistent, 16 warps in four groups:
//   warps 0-3    producer (warp 0): TMA of the CTA's own 128 rows of A and of
//                B and bulk copies of the scale tiles, five stages; MMA issuer
//                (warp 1, leader CTA only): M = 256, N = 256 pair MMAs;
//   warps 4-7    scale warps: scale tiles from shared to tensor memory;
//   warps 8-15   epilogue: two warps per 32-lane quarter.
// The accumulator fills half of tensor memory and the scales most of the rest,
// so it is not double-buffered: the epilogue's first duty is to give it back.
// setmaxnreg moves registers to the epilogue warps (80 + 96 + 168 + 168 = 4 x
// 128 per thread at launch), which lets them take all 128 accumulator columns
// into registers, hand the accumulator back, and compute and store while the
// next tile's MMAs run.
// Measured: GATED, 8192 x 5120 by 10240 + 10240, 352 us without G | U (4.9
// PFLOP/s, the rate of the plain GEMM) and 380 with it; 1777 rows 88 us, tensor
// pipe 58%.  ADAPTER, 8192 x 8192 x 8192, rank 64, eight adapters: 221 us (215
// with V in one BF16 term).
// Every mbarrier wait is bounded, as in gemm.cu.
#define NVFP4_UNIT_ERROR_WORD   // compiled without relocatable device code, for setmaxnreg
#include "tile.cuh"

namespace nvfp4 {

namespace {

enum { kGated = 0, kAdapter = 1 };

constexpr int STAGES = 5, KB_PER_STAGE = 4;
constexpr uint32_t A_BYTES = 128 * 128, B_BYTES = 128 * 128;      // 128 rows x 128 bytes, 128-byte swizzle
constexpr uint32_t SFA_BYTES = KB_PER_STAGE * 512, SFB_BYTES = 2 * KB_PER_STAGE * 512;
constexpr uint32_t OFF_A = 0;
constexpr uint32_t OFF_B = OFF_A + STAGES * A_BYTES;
constexpr uint32_t OFF_SFA = OFF_B + STAGES * B_BYTES;
constexpr uint32_t OFF_SFB = OFF_SFA + STAGES * SFA_BYTES;
constexpr uint32_t STG_BYTES = 32 * 128;                          // a 32-row x 64-column BF16 box per epilogue warp
constexpr uint32_t OFF_STG = OFF_SFB + STAGES * SFB_BYTES;
constexpr int EPI_WARPS = 8, EPI_WARP0 = 8, SF_WARPS = 4, THREADS = 512;
constexpr uint32_t OFF_BAR = OFF_STG + EPI_WARPS * STG_BYTES;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;
static_assert(OFF_STG % 1024 == 0, "swizzled boxes start on 1024 bytes");
static_assert(SMEM_BYTES <= 232448, "shared memory per block");
constexpr uint32_t TMEM_COLS = 512, ACC_COL = 0, SF_COL = 256, SF_BUF_COLS = 48, SFB_OFF = 16;

// E2M1 x E2M1, UE4M3 block scales (kind::mxf4nvf4), M = 256, N = 256.
constexpr uint32_t IDESC_FP4 = (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
// BF16 x BF16 -> FP32 (kind::f16), both K-major, M = 256, N = 256.
constexpr uint32_t IDESC_BF16 = (1u << 4) | (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | ((256u >> 4) << 24);

struct Params {
  const uint8_t* sfa;
  const uint8_t* sfb;
  const float* gsa;
  const float* gsb;
  int M, N, K;          // N: rows of B (2F for GATED)
  int group_m;
  // GATED
  int save_gu;
  float* amax_out;
  // ADAPTER: what lora.cu prepared for each 256-row tile (see AdapterPlan)
  const int* tile_count;
  const int* tile_base;
  const int* slab_adapter;
  const int* valid_rows;
  int rank, rank_blocks;   // K steps for each slab: 32 ranks each
  const int* tile_direct;
  const float* V;
  const int* row_adapter;
  const __nv_bfloat16* B;
  __nv_bfloat16* Y;
  int64_t ldy;
};

__device__ __forceinline__ void tile_at(int t, int num_m, int num_n, int group_m, int* tm, int* tn) {
  const int per_group = group_m * num_n, grp = t / per_group, first_m = grp * group_m;
  const int gsize = min(num_m - first_m, group_m), within = t - grp * per_group;
  *tm = first_m + within % gsize;
  *tn = within / gsize;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// ADAPTER: slabs that row tile tm adds to its accumulator.
__device__ __forceinline__ int tile_slabs(const Params& p, int tm) { return p.tile_direct[tm] ? 0 : p.tile_count[tm]; }

// ADAPTER, a tile without slabs: 128 columns of 32 rows, y = alpha acc + V B^T
// in FP32, eight columns at a time.  Warp-wide.
__device__ __noinline__ void direct_tile(const Params& p, uint32_t acc, float alpha, int row, int M, int col0) {
  const int id = row < M ? p.row_adapter[row] : -1;
  const float* v = p.V + static_cast<int64_t>(row) * p.rank;
#pragma unroll 1
  for (int c = 0; c < 128; c += 8) {
    uint32_t r[8];
    tmem_ld_32x32b_x8(acc + c, r);
    tmem_ld_wait();
    const int col = col0 + c;
    if (row < M && col < p.N) {
      float low[8] = {};
      const __nv_bfloat16* b = p.B + (static_cast<int64_t>(id) * p.N + col) * p.rank;
#pragma unroll 1
      for (int j = 0; id >= 0 && j < p.rank; j += 8) {
        const float4 v0 = *reinterpret_cast<const float4*>(v + j), v1 = *reinterpret_cast<const float4*>(v + j + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 w = *reinterpret_cast<const uint4*>(b + e * p.rank + j);
          const float2 w0 = bf16x2_to_f32x2(w.x), w1 = bf16x2_to_f32x2(w.y), w2 = bf16x2_to_f32x2(w.z),
                       w3 = bf16x2_to_f32x2(w.w);
          low[e] = __fmaf_rn(v0.y, w0.y, __fmaf_rn(v0.x, w0.x, low[e]));
          low[e] = __fmaf_rn(v0.w, w1.y, __fmaf_rn(v0.z, w1.x, low[e]));
          low[e] = __fmaf_rn(v1.y, w2.y, __fmaf_rn(v1.x, w2.x, low[e]));
          low[e] = __fmaf_rn(v1.w, w3.y, __fmaf_rn(v1.z, w3.x, low[e]));
        }
      }
      auto y = [&](int e) { return __fmaf_rn(__uint_as_float(r[e]), alpha, low[e]); };
      *reinterpret_cast<uint4*>(p.Y + static_cast<int64_t>(row) * p.ldy + col) =
          make_uint4(pack_bf16(y(0), y(1)), pack_bf16(y(2), y(3)), pack_bf16(y(4), y(5)), pack_bf16(y(6), y(7)));
    }
    __syncwarp();
  }
}

template <int KIND, int ACT>
__global__ void __launch_bounds__(THREADS, 1)
project_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmE,
                    const __grid_constant__ CUtensorMap tmF, const __grid_constant__ Params p) {
  // tmD: H or Y.  GATED: tmE = G | U.  ADAPTER: tmE = slabs, tmF = adapter rows [count * N, rank].
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);   // leader: A/B bytes of both CTAs
  uint64_t* empty = full + STAGES;                                 // both: leader's commit
  uint64_t* sfd_full = empty + STAGES;                             // both: own scale bytes landed
  uint64_t* sf_full = sfd_full + STAGES;                           // leader: 8 scale warps done
  uint64_t* acc_full = sf_full + STAGES;                           // both: leader's commit
  uint64_t* acc_empty = acc_full + 1;                              // leader: 16 epilogue warps
  uint64_t* mma_done = acc_empty + 1;                              // leader
  uint64_t* kind_done = mma_done + 1;                              // leader: FP4 steps of the tile finished
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(kind_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  const int sf_rows_a = (p.M + 127) / 128, sf_rows_b = (p.N + 127) / 128;
  const int katoms = (p.K + 63) / 64;
  const int num_kt = (p.K + 255) / 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfd_full[s], 1);
      mbar_init(&sf_full[s], 2 * SF_WARPS);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * EPI_WARPS);
    mbar_init(mma_done, 1);
    mbar_init(kind_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmD);
    prefetch_tmap(&tmE);
    if (KIND == kAdapter) prefetch_tmap(&tmF);
  }
  if (warp == 1) tmem_alloc_pair(const_cast<uint32_t*>(tmem_slot), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_previous_kernel();   // nothing above touches global memory
  allow_next_kernel();
  const int M = KIND == kAdapter ? min(p.M, *p.valid_rows) : p.M;
  const int num_m = (M + 255) / 256, num_n = KIND == kGated ? p.N / 256 : (p.N + 255) / 256;
  const int num_tiles = num_m * num_n;
  const uint32_t full_l = mapa_shared(smem_u32(full), 0), sf_full_l = mapa_shared(smem_u32(sf_full), 0);
  const uint32_t acc_empty_l = mapa_shared(smem_u32(acc_empty), 0);

  if (warp < 4) {
    regs_release<80>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;   // bit s: stage s holds a copy, of that parity
      for (int t = pair; t < num_tiles && !*abort_flag; t += num_pairs) {
        int tm, tn;
        tile_at(t, num_m, num_n, p.group_m, &tm, &tn);
        const int row_a = tm * 256 + 128 * static_cast<int>(rank);
        const int row_b = KIND == kGated ? tn * 128 + (p.N / 2) * static_cast<int>(rank)
                                         : tn * 256 + 128 * static_cast<int>(rank);
        const int64_t blk_a = min(2 * tm + static_cast<int>(rank), sf_rows_a - 1);
        const int64_t blk_b0 = KIND == kGated ? tn : min(2 * tn, sf_rows_b - 1);
        const int64_t blk_b1 = KIND == kGated ? sf_rows_b / 2 + tn : min(2 * tn + 1, sf_rows_b - 1);
        bool ok = true;
        for (int kt = 0; kt < num_kt; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, kErrWaitEmpty)) { ok = false; break; }
          const uint32_t sf_bytes = static_cast<uint32_t>(min(KB_PER_STAGE, katoms - kt * KB_PER_STAGE)) * 512u;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (A_BYTES + B_BYTES));
          tma_load_2d_pair(smem + OFF_A + stage * A_BYTES, &tmA, full_l + stage * 8, kt * 128, row_a);
          tma_load_2d_pair(smem + OFF_B + stage * B_BYTES, &tmB, full_l + stage * 8, kt * 128, row_b);
          mbar_arrive_expect_tx(&sfd_full[stage], 3 * sf_bytes);
          bulk_load(smem + OFF_SFA + stage * SFA_BYTES, p.sfa + (blk_a * katoms + kt * KB_PER_STAGE) * 512, sf_bytes,
                    &sfd_full[stage]);
          bulk_load(smem + OFF_SFB + stage * SFB_BYTES, p.sfb + (blk_b0 * katoms + kt * KB_PER_STAGE) * 512, sf_bytes,
                    &sfd_full[stage]);
          bulk_load(smem + OFF_SFB + stage * SFB_BYTES + KB_PER_STAGE * 512,
                    p.sfb + (blk_b1 * katoms + kt * KB_PER_STAGE) * 512, sf_bytes, &sfd_full[stage]);
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (KIND == kAdapter && ok) {
          const int count = tile_slabs(p, tm), base = p.tile_base[tm];
          for (int e = 0; e < count && ok; ++e) {
            const int row_v = (base + e) * 256 + 128 * static_cast<int>(rank);
            const int row_ad = p.slab_adapter[base + e] * p.N + row_b;
            for (int rb = 0; rb < p.rank_blocks; ++rb) {
              if (!mbar_wait(&empty[stage], phase ^ 1u, kErrWaitEmpty)) { ok = false; break; }
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (A_BYTES + B_BYTES));
              tma_load_2d_pair(smem + OFF_A + stage * A_BYTES, &tmE, full_l + stage * 8, 64 * rb, row_v);
              tma_load_2d_pair(smem + OFF_B + stage * B_BYTES, &tmF, full_l + stage * 8, 32 * rb, row_ad);
              mbar_arrive(&sfd_full[stage]);   // no scales in this step
              issued |= 1u << stage;
              issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
              if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
          }
        }
        if (!ok) { *abort_flag = 1; break; }
      }
      // Let every copy this thread started land before the CTA can exit.
      for (int s = 0; s < STAGES; ++s)
        if (issued >> s & 1u) {
          mbar_wait(&sfd_full[s], issued_parity >> s & 1u, kErrWaitFull);
          if (rank == 0) mbar_wait_cluster(&full[s], issued_parity >> s & 1u, kErrWaitFull);
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------------------------------------------------- MMA issuer (leader only)
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0, kind_phase = 0;
      const uint64_t adesc0 = smem_desc(smem_u32(smem + OFF_A), 16, 1024, 2);
      const uint64_t bdesc0 = smem_desc(smem_u32(smem + OFF_B), 16, 1024, 2);
      for (int t = pair; t < num_tiles && !*abort_flag; t += num_pairs) {
        int count = 0;
        if (KIND == kAdapter) {
          int tm, tn;
          tile_at(t, num_m, num_n, p.group_m, &tm, &tn);
          count = tile_slabs(p, tm) * p.rank_blocks;
        }
        if (!mbar_wait_cluster(acc_empty, acc_phase ^ 1u, kErrWaitAccEmpty)) { *abort_flag = 1; break; }
        tc_fence_after();
        bool ok = true;
        for (int kt = 0; kt < num_kt; ++kt) {
          if (!mbar_wait_cluster(&sf_full[stage], phase, kErrWaitFull)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sfa_t = tmem + SF_COL + stage * SF_BUF_COLS, sfb_t = sfa_t + SFB_OFF;
          const uint64_t adesc = adesc0 + static_cast<uint64_t>(stage * (A_BYTES >> 4));
          const uint64_t bdesc = bdesc0 + static_cast<uint64_t>(stage * (B_BYTES >> 4));
          if ((kt + 1) * KB_PER_STAGE <= katoms) {
#pragma unroll
            for (int kb = 0; kb < KB_PER_STAGE; ++kb)
              mma_nvf4_pair(tmem + ACC_COL, adesc + 2 * kb, bdesc + 2 * kb, IDESC_FP4, sfa_t + 4 * kb, sfb_t + 8 * kb,
                            (kt | kb) != 0);
          } else {
            const int nkb = katoms - kt * KB_PER_STAGE;
            for (int kb = 0; kb < nkb; ++kb)
              mma_nvf4_pair(tmem + ACC_COL, adesc + 2 * kb, bdesc + 2 * kb, IDESC_FP4, sfa_t + 4 * kb, sfb_t + 8 * kb,
                            (kt | kb) != 0);
          }
          tc_commit_pair_mc(&empty[stage], 0x3);
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (KIND == kAdapter && ok && count > 0) {
          // only MMAs of one kind are ordered among themselves: the FP4 steps
          // finish before a BF16 step adds to the same accumulator
          tc_commit_pair(kind_done);
          if (!mbar_wait(kind_done, kind_phase, kErrWaitAccFull)) { *abort_flag = 1; break; }
          kind_phase ^= 1u;
          tc_fence_after();
          int ranks = p.rank;   // left of the slab under way
          for (int e = 0; e < count; ++e) {
            if (!mbar_wait_cluster(&sf_full[stage], phase, kErrWaitFull)) { ok = false; break; }
            tc_fence_after();
            const uint64_t adesc = adesc0 + static_cast<uint64_t>(stage * (A_BYTES >> 4));
            const uint64_t bdesc = bdesc0 + static_cast<uint64_t>(stage * (B_BYTES >> 4));
            // columns 0-31 of the slab's step: first terms, 32-63: second (4 x 16 bytes on); 16 ranks an MMA
            mma_bf16_pair(tmem + ACC_COL, adesc, bdesc, IDESC_BF16, 1);
            mma_bf16_pair(tmem + ACC_COL, adesc + 4, bdesc, IDESC_BF16, 1);
            if (ranks > 16) {
              mma_bf16_pair(tmem + ACC_COL, adesc + 2, bdesc + 2, IDESC_BF16, 1);
              mma_bf16_pair(tmem + ACC_COL, adesc + 6, bdesc + 2, IDESC_BF16, 1);
            }
            if ((ranks -= 32) <= 0) ranks = p.rank;
            tc_commit_pair_mc(&empty[stage], 0x3);
            if (++stage == STAGES) stage = 0, phase ^= 1u;
          }
        }
        if (!ok) { *abort_flag = 1; break; }
        tc_commit_pair_mc(acc_full, 0x3);
        acc_phase ^= 1u;
      }
      tc_commit_pair(mma_done);
      mbar_wait(mma_done, 0, kErrWaitAccFull);
    }
  } else if (warp < EPI_WARP0) {
    regs_release<96>();
    // ------------------------------------------------------------ scale warps (both CTAs)
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    for (int t = pair; t < num_tiles && !*abort_flag; t += num_pairs) {
      int tm, tn;
      tile_at(t, num_m, num_n, p.group_m, &tm, &tn);
      const bool a_sf = 2 * tm + static_cast<int>(rank) < sf_rows_a;
      const bool b_sf0 = KIND == kGated || 2 * tn < sf_rows_b, b_sf1 = KIND == kGated || 2 * tn + 1 < sf_rows_b;
      const int extra = KIND == kAdapter ? tile_slabs(p, tm) * p.rank_blocks : 0;
      bool ok = true;
      for (int kt = 0; kt < num_kt + extra; ++kt) {
        if (!mbar_wait(&sfd_full[stage], phase, kErrWaitFull) ||
            (rank == 0 && !mbar_wait_cluster(&full[stage], phase, kErrWaitFull))) {
          ok = false;
          break;
        }
        if (kt < num_kt) {
          const int nkb = min(KB_PER_STAGE, katoms - kt * KB_PER_STAGE);
          const uint8_t* sa = smem + OFF_SFA + stage * SFA_BYTES + lane * 16;
          const uint8_t* sb = smem + OFF_SFB + stage * SFB_BYTES + lane * 16;
          uint32_t ra[16], rb[32];
          const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int kb = 0; kb < KB_PER_STAGE; ++kb) {
            const uint4 va = kb < nkb && a_sf ? *reinterpret_cast<const uint4*>(sa + 512 * kb) : zero;
            const uint4 v0 = kb < nkb && b_sf0 ? *reinterpret_cast<const uint4*>(sb + 512 * kb) : zero;
            const uint4 v1 =
                kb < nkb && b_sf1 ? *reinterpret_cast<const uint4*>(sb + KB_PER_STAGE * 512 + 512 * kb) : zero;
            ra[4 * kb + 0] = va.x; ra[4 * kb + 1] = va.y; ra[4 * kb + 2] = va.z; ra[4 * kb + 3] = va.w;
            rb[8 * kb + 0] = v0.x; rb[8 * kb + 1] = v0.y; rb[8 * kb + 2] = v0.z; rb[8 * kb + 3] = v0.w;
            rb[8 * kb + 4] = v1.x; rb[8 * kb + 5] = v1.y; rb[8 * kb + 6] = v1.z; rb[8 * kb + 7] = v1.w;
          }
          const uint32_t sfa_t = tmem + lane_base + SF_COL + stage * SF_BUF_COLS;
          tmem_st_32x32b_x16(sfa_t, ra);
          tmem_st_32x32b_x32(sfa_t + SFB_OFF, rb);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(sf_full_l + stage * 8);
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
      if (!ok) { *abort_flag = 1; break; }
    }
  } else {
    regs_claim<168>();
    // ------------------------------------------------------------ epilogue (both CTAs)
    // Boxes of 32 rows x 64 BF16 columns leave through shared memory and TMA:
    // row r's 16-byte chunk j sits at r * 128 + 16 (j ^ (r % 8)), the 128-byte
    // swizzle that the output maps name.
    const int quarter = warp & 3, half = (warp - EPI_WARP0) >> 2;
    const float alpha = __fmul_rn(*p.gsa, *p.gsb);
    const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + ACC_COL;
    uint8_t* stg = smem + OFF_STG + (warp - EPI_WARP0) * STG_BYTES;
    uint8_t* my_row = stg + lane * 128;
    const int sw = lane & 7;
    // chunk(j): columns 8 j .. 8 j + 7 of the lane's row, packed
    auto box_out = [&](const CUtensorMap* tm, int col, int row0, auto&& chunk) {
      if (lane == 0) bulk_wait_read_all();   // the previous box has left the staging buffer
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(my_row + 16 * (j ^ sw)) = chunk(j);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tm, stg, col, row0);
        bulk_commit_group();
      }
    };
    uint32_t acc_phase = 0;
    float run_max = 0.0f;
    for (int t = pair; t < num_tiles && !*abort_flag; t += num_pairs) {
      int tm, tn;
      tile_at(t, num_m, num_n, p.group_m, &tm, &tn);
      const bool direct = KIND == kAdapter && p.tile_direct[tm];
      if (!mbar_wait_cluster(acc_full, acc_phase, kErrWaitAccFull)) { *abort_flag = 1; break; }
      acc_phase ^= 1u;
      tc_fence_after();
      const int row0 = tm * 256 + 128 * static_cast<int>(rank) + quarter * 32;
      if (KIND == kGated) {
        // this warp's 64 columns of G (accumulator columns 64 half ..) and of U (128 + 64 half ..)
        uint32_t g[2][32], u[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tmem_ld_32x32b_x32(acc + 64 * half + 32 * c, g[c]);
          tmem_ld_32x32b_x32(acc + 128 + 64 * half + 32 * c, u[c]);
        }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_l);
        if (row0 < M) {
          const int col0 = tn * 128 + 64 * half;
          if (p.save_gu) {
            auto scaled = [&](const uint32_t (&v)[2][32], int j) {
              const uint32_t* x = &v[j >> 2][8 * (j & 3)];
              auto f = [&](int i) { return __uint_as_float(x[i]) * alpha; };
              return make_uint4(pack_bf16(f(0), f(1)), pack_bf16(f(2), f(3)), pack_bf16(f(4), f(5)), pack_bf16(f(6), f(7)));
            };
            box_out(&tmE, col0, row0, [&](int j) { return scaled(g, j); });
            box_out(&tmE, p.N / 2 + col0, row0, [&](int j) { return scaled(u, j); });
          }
          float tile_max = 0.0f;
          box_out(&tmD, col0, row0, [&](int j) {
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float gv = __uint_as_float(g[j >> 2][8 * (j & 3) + i]) * alpha;
              const float uv = __uint_as_float(u[j >> 2][8 * (j & 3) + i]) * alpha;
              h[i] = gv * gate_sigmoid<ACT>(gv) * uv;
              tile_max = fmaxf(tile_max, fabsf(h[i]));
            }
            return make_uint4(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]), pack_bf16(h[4], h[5]), pack_bf16(h[6], h[7]));
          });
          if (row0 + lane < M) run_max = fmaxf(run_max, tile_max);
        }
      } else if (direct) {
        direct_tile(p, acc + 128 * half, alpha, row0 + lane, M, tn * 256 + 128 * half);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_l);
      } else {
        uint32_t w[2][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(acc + 128 * half + 32 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[c >> 1][16 * (c & 1) + e] = pack_bf16(__uint_as_float(r[2 * e]) * alpha, __uint_as_float(r[2 * e + 1]) * alpha);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = tn * 256 + 128 * half + 64 * h;
          if (row0 >= M || col >= p.N) continue;
          if (row0 + 32 <= M) {
            box_out(&tmD, col, row0, [&](int j) {
              return make_uint4(w[h][4 * j], w[h][4 * j + 1], w[h][4 * j + 2], w[h][4 * j + 3]);
            });
          } else if (row0 + lane < M) {   // the rows from M on stay as they are: plain stores
            uint4* dst = reinterpret_cast<uint4*>(p.Y + static_cast<int64_t>(row0 + lane) * p.ldy + col);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + 8 * j < p.N) dst[j] = make_uint4(w[h][4 * j], w[h][4 * j + 1], w[h][4 * j + 2], w[h][4 * j + 3]);
          }
          __syncwarp();
        }
      }
    }
    if (KIND == kGated && p.amax_out) {
      // max |H| as stored: one rounding of the largest |h| is the largest rounded |h|
      const unsigned int here = __activemask();
      const uint32_t v = __reduce_max_sync(here, __float_as_uint(__bfloat162float(__float2bfloat16_rn(run_max))));
      if (lane == __ffs(here) - 1 && v != 0u) atomicMax(reinterpret_cast<unsigned int*>(p.amax_out), v);
    }
    if (lane == 0) bulk_wait_all();  // stores complete before the CTA's shared memory goes away
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal its barriers
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, TMEM_COLS);
}

template <class Kernel>
cudaError_t launch_pairs(Kernel kern, SmemOptIn* opt, int64_t tiles, int num_sms, cudaStream_t s, const CUtensorMap& a,
                         const CUtensorMap& b, const CUtensorMap& d, const CUtensorMap& e, const CUtensorMap& f,
                         Params p) {
  cudaError_t err = opt->ensure(kern, SMEM_BYTES);
  if (err != cudaSuccess) return err;
  const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  // Raster group: as many M-tiles (8, 16 or 32) as keep their rows of A within
  // 32 MB of L2 while the group walks all of N.
  p.group_m = 8;
  while (p.group_m < 32 && 2LL * p.group_m * 256 * (p.K / 2) <= (32LL << 20)) p.group_m *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, b, d, e, f, p);
}

SmemOptIn g_opt_silu, g_opt_gelu, g_opt_adapter;

}  // namespace

cudaError_t read_project_error(unsigned int* out, int clear) { return read_unit_error(out, clear); }

cudaError_t launch_gated_tiles(const FpOperand& a, const FpOperand& w, int64_t M, int64_t F, int64_t K, int act, void* H,
                               int64_t ldh, void* GU, float* amax_out, int num_sms, cudaStream_t s) {
  CUtensorMap tmA, tmB, tmD, tmE;
  if (!operand_map(&tmA, a.data, M, K, 128) || !operand_map(&tmB, w.data, 2 * F, K, 128) ||
      !bf16_map(&tmD, H, M, F, ldh, 32) || !bf16_map(&tmE, GU ? GU : H, M, GU ? 2 * F : F, GU ? 2 * F : ldh, 32))
    return cudaErrorInvalidValue;
  if (amax_out) {
    cudaError_t e = launch_zero(amax_out, 1, s);
    if (e != cudaSuccess) return e;
  }
  Params p = {};
  p.sfa = a.scales;
  p.sfb = w.scales;
  p.gsa = a.gs;
  p.gsb = w.gs;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(2 * F);
  p.K = static_cast<int>(K);
  p.save_gu = GU != nullptr;
  p.amax_out = amax_out;
  const int64_t tiles = ((M + 255) / 256) * (F / 128);
  return act ? launch_pairs(project_pair_kernel<kGated, 1>, &g_opt_gelu, tiles, num_sms, s, tmA, tmB, tmD, tmE, tmE, p)
             : launch_pairs(project_pair_kernel<kGated, 0>, &g_opt_silu, tiles, num_sms, s, tmA, tmB, tmD, tmE, tmE, p);
}

cudaError_t launch_adapter_tiles(const FpOperand& a, const FpOperand& w, int64_t M, int64_t N, int64_t K,
                                 const AdapterPlan& plan, const void* adapter_rows, int64_t adapters, int64_t rank,
                                 void* Y, int64_t ldy, int num_sms, cudaStream_t s) {
  const int64_t rank_blocks = (rank + 31) / 32;
  CUtensorMap tmA, tmB, tmD, tmE, tmF;
  if (!operand_map(&tmA, a.data, M, K, 128) || !operand_map(&tmB, w.data, N, K, 128) ||
      !bf16_map(&tmD, Y, M, N, ldy, 32) || !bf16_map(&tmE, plan.slabs, plan.max_slabs * 256, rank_blocks * 64, rank_blocks * 64, 128) ||
      !bf16_map(&tmF, adapter_rows, adapters * N, rank, rank, 128))
    return cudaErrorInvalidValue;
  Params p = {};
  p.sfa = a.scales;
  p.sfb = w.scales;
  p.gsa = a.gs;
  p.gsb = w.gs;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.tile_count = plan.tile_count;
  p.tile_base = plan.tile_base;
  p.slab_adapter = plan.slab_adapter;
  p.valid_rows = plan.valid_rows;
  p.rank = static_cast<int>(rank);
  p.tile_direct = plan.tile_direct;
  p.V = plan.V;
  p.row_adapter = plan.row_adapter;
  p.B = static_cast<const __nv_bfloat16*>(adapter_rows);
  p.rank_blocks = static_cast<int>(rank_blocks);
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.ldy = ldy;
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  return launch_pairs(project_pair_kernel<kAdapter, 0>, &g_opt_adapter, tiles, num_sms, s, tmA, tmB, tmD, tmE, tmF, p);
}

}  // namespace nvfp4
