// rows.cu -- FP4 projections of few rows (serving: single tokens, decode
// batches), and the quantizer in front of them.
//
// With T <= 128 rows of X the work is reading W once: 0.5625 bytes for each of
// its elements.  The roles of the operands are therefore swapped: a tile is
// 128 rows of W (the MMA's M) by all T rows of X (its N, padded to 16), so no
// part of a tile is padding in the operand that costs bandwidth.
//
//   GATED    a tile holds 64 gate rows and the 64 up rows that belong to them
//            (two TMA boxes in one operand tile; the scale warps pick the
//            matching halves of two scale tiles);
//   ADAPTER  a tile holds 128 output channels; the epilogue adds
//            sum_j V[t, j] B_i[n, j] for the adapter i of row t.
//
// One CTA for each tile and slice of K.  Where there are fewer tiles than fill
// the GPU, a cluster of 2, 4 or 8 CTAs splits K; its partial tiles meet in
// shared memory (distributed shared memory, summed in CTA order: the result
// does not depend on timing).  Two CTAs share an SM.
//   warps 0, 10  producers: TMA of the W and the X tiles, bulk copies of their
//                scales (a thread issues a copy in about 50 ns, and a step has
//                five or six: one producer for all was the stream's limit);
//   warp 1       MMA issuer: M = 128, N = 16 .. 128, K = 64 a step;
//   warps 2-5    scale warps, then the accumulator's way to shared memory;
//   warps 6-9    output; for ADAPTER they compute the low-rank sums of their
//                channel while W streams, up to 32 rows of X for each CTA, and
//                keep them in shared memory (done after the loop, the sums of
//                64 rows took twice as long as the loop); then they and warps
//                2-5 write the output.
// Measured, quantizer included: GATED, 5120 by 10240 + 10240 (59 MB of W), one
// row 16.4 us, 48 rows 19.3 us; ADAPTER, 8192 x 8192, rank 16, 64 requests of
// one row 19.3 us.  The kernel itself reads DRAM at 2.2 to 2.7 TB/s under ncu,
// from a cold start to the last output; the rest is the quantizer in front (4
// us).  The gated case has 160 tiles in one slice each: 160 CTAs for 296 places,
// each walking 20 K steps through one chain of scales, MMA and commit.
// W does not depend on the kernel before this one (the quantizer of X), so the
// producer fills the ring with W before it waits for that kernel to finish
// (programmatic dependent launch).
#define NVFP4_UNIT_ERROR_WORD
#include "lowrank.cuh"
#include "tile.cuh"

namespace nvfp4 {

namespace {

enum { kGated = 0, kAdapter = 1 };
constexpr int KB_PER_STAGE = 4, THREADS = 352, MAX_STAGES = 5, OUT_WARP0 = 6, X_WARP = 10, KEEP = 32;
constexpr uint32_t A_BYTES = 128 * 128, SF_BYTES = KB_PER_STAGE * 512;

struct RowsParams {
  const uint8_t* sfw;
  const uint8_t* sfx;
  const float* gsw;
  const float* gsx;
  int T, N, K;             // rows of X, rows of W (2F for GATED), contraction
  int tile0;               // the launch's first tile
  int n_pad, stages, slices, keep;   // keep: rows of X whose low-rank sums are made beside the loop
  uint32_t tmem_cols, b_bytes;
  __nv_bfloat16* out;      // [T, F] or [T, N]
  int64_t ldo;
  // ADAPTER
  const float* V;          // [T, rank]
  const int* row_adapter;  // [T]; -1 none, -2 padding row (left alone)
  const __nv_bfloat16* B;  // [adapters, N, rank]
  int rank;
};

template <int KIND, int ACT>
__global__ void __launch_bounds__(THREADS)
project_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ RowsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  allow_next_kernel();   // the launch of the last tiles
  __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], sf_full[MAX_STAGES], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int ids[KEEP];   // ADAPTER: the adapters of a pass's rows of X
  // ring: W tiles, X tiles, then W's scale tiles (two for GATED) and X's
  constexpr uint32_t SFW_BYTES = (KIND == kGated ? 2 : 1) * SF_BYTES;
  uint8_t* w_ring = smem;
  uint8_t* x_ring = w_ring + p.stages * A_BYTES;
  uint8_t* sfw_ring = x_ring + p.stages * p.b_bytes;
  uint8_t* sfx_ring = sfw_ring + p.stages * SFW_BYTES;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = p.slices, slice = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = p.tile0 + blockIdx.x / slices;
  const int katoms = p.K / 64, num_kt = (katoms + KB_PER_STAGE - 1) / KB_PER_STAGE;
  const int kt0 = num_kt * slice / slices, nk = num_kt * (slice + 1) / slices - kt0;
  // rows of W in this tile: [row0, +64) and [row1, +64)
  const int row0 = KIND == kGated ? tile * 64 : tile * 128, row1 = KIND == kGated ? p.N / 2 + row0 : row0 + 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 2);   // both producers
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 4);
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t sf_col = (p.n_pad + 31) / 32 * 32;   // accumulator first, then 32 scale columns a stage

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer of W
    int stage = 0, last = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nk; ++i) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, kErrWaitEmpty)) break;
      const int kt = kt0 + i;
      const uint32_t sf = static_cast<uint32_t>(min(KB_PER_STAGE, katoms - kt * KB_PER_STAGE)) * 512u;
      mbar_arrive_expect_tx(&full[stage], A_BYTES + (KIND == kGated ? 2 : 1) * sf);
      tma_load_2d(w_ring + stage * A_BYTES, &tmW, &full[stage], kt * 128, row0);
      if (KIND == kGated) tma_load_2d(w_ring + stage * A_BYTES + A_BYTES / 2, &tmW, &full[stage], kt * 128, row1);
      const int64_t b0 = row0 >> 7, b1 = row1 >> 7;
      bulk_load(sfw_ring + stage * SFW_BYTES, p.sfw + (b0 * katoms + kt * KB_PER_STAGE) * 512, sf, &full[stage]);
      if (KIND == kGated)
        bulk_load(sfw_ring + stage * SFW_BYTES + SF_BYTES, p.sfw + (b1 * katoms + kt * KB_PER_STAGE) * 512, sf, &full[stage]);
      last = i + 1;
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
    // let every copy land before shared memory is reused or given up
    for (int i = max(0, last - p.stages); i < last; ++i)
      mbar_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, kErrWaitFull);
  } else if (warp == X_WARP && lane == 0) {
    // ------------------------------------------------------------ producer of X
    wait_previous_kernel();
    int stage = 0, last = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nk; ++i) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, kErrWaitEmpty)) break;
      const int kt = kt0 + i;
      const uint32_t sf = static_cast<uint32_t>(min(KB_PER_STAGE, katoms - kt * KB_PER_STAGE)) * 512u;
      mbar_arrive_expect_tx(&full[stage], p.b_bytes + sf);
      tma_load_2d(x_ring + stage * p.b_bytes, &tmX, &full[stage], kt * 128, 0);
      bulk_load(sfx_ring + stage * SF_BYTES, p.sfx + static_cast<int64_t>(kt * KB_PER_STAGE) * 512, sf, &full[stage]);
      last = i + 1;
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
    for (int i = max(0, last - p.stages); i < last; ++i)
      mbar_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, kErrWaitFull);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc =
        (1u << 7) | (1u << 10) | (static_cast<uint32_t>(p.n_pad >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
    const uint64_t adesc0 = smem_desc(smem_u32(w_ring), 16, 1024, 2), bdesc0 = smem_desc(smem_u32(x_ring), 16, 1024, 2);
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nk; ++i) {
      if (!mbar_wait(&sf_full[stage], phase, kErrWaitFull)) break;
      tc_fence_after();
      const int nkb = min(KB_PER_STAGE, katoms - (kt0 + i) * KB_PER_STAGE);
      const uint64_t adesc = adesc0 + static_cast<uint64_t>(stage * (A_BYTES >> 4));
      const uint64_t bdesc = bdesc0 + static_cast<uint64_t>(stage * (p.b_bytes >> 4));
      const uint32_t sfa_t = tmem + sf_col + stage * 32;
      for (int kb = 0; kb < nkb; ++kb)
        mma_nvf4(tmem, adesc + 2 * kb, bdesc + 2 * kb, idesc, sfa_t + 4 * kb, sfa_t + 16 + 4 * kb, (i | kb) != 0);
      tc_commit(&empty[stage]);
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
    tc_commit(&acc_full);   // completes when every MMA issued so far has
    mbar_wait(&acc_full, 0, kErrWaitAccFull);
  } else if (warp >= 2 && warp < OUT_WARP0) {
    // ------------------------------------------------------------ scale warps
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int h0 = (row0 >> 6) & 1, h1 = (row1 >> 6) & 1;   // GATED: halves of the two scale tiles
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nk; ++i) {
      if (!mbar_wait(&full[stage], phase, kErrWaitFull)) break;
      const int nkb = min(KB_PER_STAGE, katoms - (kt0 + i) * KB_PER_STAGE);
      const uint8_t* sw = sfw_ring + stage * SFW_BYTES + lane * 16;
      const uint8_t* sx = sfx_ring + stage * SF_BYTES + lane * 16;
      uint32_t r[32];
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int kb = 0; kb < KB_PER_STAGE; ++kb) {
        uint4 v = zero;
        if (kb < nkb) {
          if (KIND == kGated) {
            const uint2 g = *reinterpret_cast<const uint2*>(sw + 512 * kb + 8 * h0);
            const uint2 u = *reinterpret_cast<const uint2*>(sw + SF_BYTES + 512 * kb + 8 * h1);
            v = make_uint4(g.x, g.y, u.x, u.y);
          } else {
            v = *reinterpret_cast<const uint4*>(sw + 512 * kb);
          }
        }
        const uint4 x = kb < nkb ? *reinterpret_cast<const uint4*>(sx + 512 * kb) : zero;
        r[4 * kb + 0] = v.x; r[4 * kb + 1] = v.y; r[4 * kb + 2] = v.z; r[4 * kb + 3] = v.w;
        r[16 + 4 * kb + 0] = x.x; r[16 + 4 * kb + 1] = x.y; r[16 + 4 * kb + 2] = x.z; r[16 + 4 * kb + 3] = x.w;
      }
      tmem_st_32x32b_x32(tmem + lane_base + sf_col + stage * 32, r);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sf_full[stage]);
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
  }
  // ADAPTER: the low-rank sums of this CTA's rows of X (t = slice + slices * i)
  // for the tile's 128 channels, a thread each, KEEP rows a pass: V and the
  // adapters of the pass go to shared memory first, then four rows' loads of B
  // (16 ranks) are in flight at a time.
  float* add = reinterpret_cast<float*>(sfx_ring + p.stages * SF_BYTES);   // [keep][128]
  float* vbuf = add + p.keep * 128;                                        // [keep][rank]
  const int ch = static_cast<int>(threadIdx.x) - 32 * OUT_WARP0;
  auto low_rank_pass = [&](int i0) {
    for (int u = ch; u < p.keep * (p.rank / 4); u += 128) {
      const int i = u / (p.rank / 4), t = slice + slices * (i0 + i);
      if (t < p.T)
        reinterpret_cast<float4*>(vbuf)[u] = *reinterpret_cast<const float4*>(
            p.V + static_cast<int64_t>(t) * p.rank + (u - i * (p.rank / 4)) * 4);
    }
    if (ch < p.keep) ids[ch] = slice + slices * (i0 + ch) < p.T ? p.row_adapter[slice + slices * (i0 + ch)] : -2;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const bool live = row0 + ch < p.N;
#pragma unroll 1
    for (int i = 0; i < p.keep; i += 4) {
      float x[4] = {};
#pragma unroll 1
      for (int k = 0; k < p.rank; k += 16) {
        uint4 w[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int id = ids[i + e];
          const uint4* b = reinterpret_cast<const uint4*>(p.B + (static_cast<int64_t>(id) * p.N + row0 + ch) * p.rank + k);
          w[e][0] = id >= 0 && live ? *b : make_uint4(0, 0, 0, 0);
          w[e][1] = id >= 0 && live && k + 8 < p.rank ? b[1] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (ids[i + e] < 0) continue;   // uniform; V of such a row is not defined
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (k + 8 * h >= p.rank) break;
            const float4* v = reinterpret_cast<const float4*>(vbuf + (i + e) * p.rank + k + 8 * h);
            const float4 v0 = v[0], v1 = v[1];
            const float2 w0 = bf16x2_to_f32x2(w[e][h].x), w1 = bf16x2_to_f32x2(w[e][h].y),
                         w2 = bf16x2_to_f32x2(w[e][h].z), w3 = bf16x2_to_f32x2(w[e][h].w);
            x[e] = __fmaf_rn(v0.x, w0.x, x[e]);
            x[e] = __fmaf_rn(v0.y, w0.y, x[e]);
            x[e] = __fmaf_rn(v0.z, w1.x, x[e]);
            x[e] = __fmaf_rn(v0.w, w1.y, x[e]);
            x[e] = __fmaf_rn(v1.x, w2.x, x[e]);
            x[e] = __fmaf_rn(v1.y, w2.y, x[e]);
            x[e] = __fmaf_rn(v1.z, w3.x, x[e]);
            x[e] = __fmaf_rn(v1.w, w3.y, x[e]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) add[(i + e) * 128 + ch] = x[e];
    }
  };
  if (KIND == kAdapter && warp >= OUT_WARP0 && warp < X_WARP) {
    wait_previous_kernel();
    low_rank_pass(0);
  }
  __syncwarp();

  // The accumulator as FP32 in shared memory: part[q][i][128 rows of W] holds
  // slice q's partial of row t = slice + slices * i of X.  Every CTA writes its
  // partials straight into the shared memory of the CTA that sums them (stores
  // need no answer, loads would wait for one).  The ring underneath is idle: the
  // accumulator is complete, so every copy was consumed, here and (after the
  // first cluster barrier) in the peers.
  float* part = reinterpret_cast<float*>(smem);
  const int mine = (p.T + slices - 1) / slices;   // rows of X a CTA sums, at most
  if (warp >= 2 && warp < OUT_WARP0) mbar_wait(&acc_full, 0, kErrWaitAccFull);
  __syncwarp();
  if (slices > 1) cluster_sync();
  if (warp >= 2 && warp < OUT_WARP0) {
    tc_fence_after();
    const int r = (warp & 3) * 32 + lane;
    const uint32_t part_addr = smem_u32(part) + (slice * mine * 128 + r) * 4;
#pragma unroll 1
    for (int c = 0; c < p.n_pad; c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c, v);
      tmem_ld_wait();
      if (slices == 1) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c + e < p.T) part[(c + e) * 128 + r] = __uint_as_float(v[e]);
      } else {
        const int shift = 31 - __clz(slices);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c + e < p.T)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                             mapa_shared(part_addr + ((c + e) >> shift) * 512, (c + e) & (slices - 1))),
                         "r"(v[e])
                         : "memory");
      }
    }
  }
  tc_fence_before();
  if (slices > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
  if (warp >= 2 && warp < X_WARP) {
    if (KIND == kGated || warp < OUT_WARP0) wait_previous_kernel();
    const float alpha = __fmul_rn(*p.gsx, __ldg(p.gsw));
    // two neighbouring rows of W (channels) of this CTA's i-th row of X
    auto sum2 = [&](int i, int row) {
      float2 acc = *reinterpret_cast<const float2*>(part + i * 128 + row);
      for (int q = 1; q < slices; ++q) {
        const float2 v = *reinterpret_cast<const float2*>(part + (q * mine + i) * 128 + row);
        acc.x += v.x;
        acc.y += v.y;
      }
      return acc;
    };
    const int u = threadIdx.x - 64;   // 0 .. 255
    if (KIND == kGated) {   // 32 channel pairs x eight rows of X at a time
      const int j = 2 * (u & 31);
#pragma unroll 2
      for (int i = u >> 5; slice + slices * i < p.T; i += 8) {
        const float2 g = sum2(i, j), v = sum2(i, 64 + j);
        const float gx = g.x * alpha, gy = g.y * alpha;
        const __nv_bfloat162 h = __floats2bfloat162_rn(gx * gate_sigmoid<ACT>(gx) * (v.x * alpha),
                                                       gy * gate_sigmoid<ACT>(gy) * (v.y * alpha));
        *reinterpret_cast<__nv_bfloat162*>(p.out + (slice + slices * i) * p.ldo + row0 + j) = h;
      }
    } else {   // 64 channel pairs x four rows of X at a time
      const int j = 2 * (u & 63);
#pragma unroll 1
      for (int i0 = 0; i0 < mine; i0 += p.keep) {
        if (i0 > 0) {   // rows beyond those done beside the loop
          asm volatile("bar.sync 2, 256;" ::: "memory");
          if (warp >= OUT_WARP0) low_rank_pass(i0);
          asm volatile("bar.sync 2, 256;" ::: "memory");
        }
#pragma unroll 2
        for (int i = u >> 6; i < p.keep && slice + slices * (i0 + i) < p.T; i += 4) {
          if (ids[i] == -2 || row0 + j >= p.N) continue;
          const float2 x = sum2(i0 + i, j);
          const float2 low = *reinterpret_cast<const float2*>(add + i * 128 + j);
          *reinterpret_cast<__nv_bfloat162*>(p.out + (slice + slices * (i0 + i)) * p.ldo + row0 + j) =
              __floats2bfloat162_rn(__fmaf_rn(x.x, alpha, low.x), __fmaf_rn(x.y, alpha, low.y));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Per-tensor amax and row-wise quantization of a few rows in one launch: one
// CTA or one cluster of CTAS.  A thread keeps its first blocks of 16 elements
// in registers, the maxima meet in every CTA's shared memory, and the same
// blocks are then scaled and rounded (the arithmetic of quantize.cu's row
// kernel, to nearest or stochastic, with its draws).
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = kRowThreads, kQuantKeep = 4;
constexpr int kMaxQuantCtas = 16;

struct QuantOut {
  uint8_t* data;
  uint8_t* sf;
  float* gs;
  int sr;
  uint32_t k0, k1;
};

template <int CTAS>
__device__ void quantize_rows_cluster(const uint16_t* __restrict__ x, int T, int C, int64_t ld,
                                      const QuantOut& out, uint32_t rank) {
  __shared__ uint32_t warp_max[kQuantThreads / 32], cta_max[CTAS];
  __shared__ float r_tbl[kRTableSize];
  const int S = C / 16, blocks = T * S, stride = CTAS * kQuantThreads;
  const int first = static_cast<int>(rank) * kQuantThreads + threadIdx.x;
  if (CTAS > 1) cluster_arrive();   // this CTA runs; its peers wait for that before they store into it
  uint4 keep[kQuantKeep][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i) {
    const int b = first + i * stride;
    keep[i][0] = keep[i][1] = make_uint4(0, 0, 0, 0);
    if (b < blocks) {
      const int r = b / S;
      const uint4* src = reinterpret_cast<const uint4*>(x + r * ld + (b - r * S) * 16);
      keep[i][0] = __ldg(src);
      keep[i][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i) m = max(m, max(absmax_bits8(keep[i][0]), absmax_bits8(keep[i][1])));
  for (int b = first + kQuantKeep * stride; b < blocks; b += stride) {
    const int r = b / S;
    const uint4* src = reinterpret_cast<const uint4*>(x + r * ld + (b - r * S) * 16);
    m = max(m, max(absmax_bits8(__ldg(src)), absmax_bits8(__ldg(src + 1))));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (CTAS > 1) cluster_wait();   // every peer's shared memory exists
  if (threadIdx.x < 32) {
    m = threadIdx.x < kQuantThreads / 32 ? warp_max[threadIdx.x] : 0u;
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (CTAS == 1) {
      if (threadIdx.x == 0) cta_max[0] = m;
    } else if (threadIdx.x < CTAS)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&cta_max[rank]), threadIdx.x)), "r"(m)
                   : "memory");
  }
  if (CTAS == 1)
    __syncthreads();
  else
    cluster_sync();
  m = 0;
#pragma unroll
  for (int q = 0; q < CTAS; ++q) m = max(m, cta_max[q]);
  const float amax = __uint_as_float(m << 16), s_enc = encode_scale(amax);
  const bool flagged = !isfinite(amax);   // as quantize.cu: NaN scales, zero codes
  if (first == 0) *out.gs = decode_scale(amax);
  fill_r_table(r_tbl, s_enc);
  __syncthreads();
  auto put = [&](int b, uint4 a, uint4 c) {
    const int r = b / S, k = b - r * S;
    float2 y[8] = {bf16x2_to_f32x2(a.x), bf16x2_to_f32x2(a.y), bf16x2_to_f32x2(a.z), bf16x2_to_f32x2(a.w),
                   bf16x2_to_f32x2(c.x), bf16x2_to_f32x2(c.y), bf16x2_to_f32x2(c.z), bf16x2_to_f32x2(c.w)};
    const uint32_t mb = max(absmax_bits8(a), absmax_bits8(c));
    BlockScale bs{0x7Fu, 0.0f};
    uint32_t w0 = 0, w1 = 0;
    if (!flagged) {
      bs = block_scale_t(bf16_bits_to_f32(mb), s_enc, r_tbl);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = make_float2(__fmul_rn(y[i].x, bs.r), __fmul_rn(y[i].y, bs.r));
      if (out.sr) {   // block counter (r C) / 16 + k
        const u32x4 w = sr_words<true>(static_cast<uint64_t>(b), kDomainRowSR, out.k0, out.k1);
        w0 = sr_e2m1x4(y[0].x, y[0].y, y[1].x, y[1].y, w.x) | (sr_e2m1x4(y[2].x, y[2].y, y[3].x, y[3].y, w.y) << 16);
        w1 = sr_e2m1x4(y[4].x, y[4].y, y[5].x, y[5].y, w.z) | (sr_e2m1x4(y[6].x, y[6].y, y[7].x, y[7].y, w.w) << 16);
      } else {
        w0 = f32x8_to_e2m1x8(y[0].x, y[0].y, y[1].x, y[1].y, y[2].x, y[2].y, y[3].x, y[3].y);
        w1 = f32x8_to_e2m1x8(y[4].x, y[4].y, y[5].x, y[5].y, y[6].x, y[6].y, y[7].x, y[7].y);
      }
      w0 = clear_negative_zero(w0);
      w1 = clear_negative_zero(w1);
    }
    *reinterpret_cast<uint2*>(out.data + static_cast<int64_t>(r) * (C / 2) + k * 8) = make_uint2(w0, w1);
    out.sf[sf_offset(r, k, S)] = static_cast<uint8_t>(bs.sf);
  };
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i) {
    const int b = first + i * stride;
    if (b < blocks) put(b, keep[i][0], keep[i][1]);
  }
  for (int b = first + kQuantKeep * stride; b < blocks; b += stride) {
    const int r = b / S;
    const uint4* src = reinterpret_cast<const uint4*>(x + r * ld + (b - r * S) * 16);
    put(b, __ldg(src), __ldg(src + 1));
  }
}

template <int CTAS>
__global__ void __launch_bounds__(kQuantThreads, 1)
quant_few_rows_kernel(const uint16_t* __restrict__ x, int T, int C, int64_t ld, QuantOut out) {
  allow_next_kernel();
  quantize_rows_cluster<CTAS>(x, T, C, ld, out, CTAS == 1 ? 0 : cluster_ctarank());
}

// The same beside V = scale_i x A_i^T for few rows: the first cluster quantizes,
// every other CTA takes one row and eight ranks, sixteen warps splitting the columns
// (an adapter is read once for each row that uses it, mostly from L2).  Two CTAs
// share an SM, as clusters of 16 otherwise leave room for 128 of them at a time
// (8192 x 8192, rank 64, 64 rows: 51.6 us with one, 46.8 with two; rank 8, 128
// rows: 26.1 and 27.4).
template <int CTAS>
__global__ void __launch_bounds__(kQuantThreads, 2)
lora_few_rows_kernel(const uint16_t* __restrict__ x, int T, int C, int64_t ld, QuantOut out, const uint16_t* A,
                     LoraBatch b, int* __restrict__ row_adapter, float* __restrict__ V) {
  allow_next_kernel();
  if (out.sr) wait_previous_kernel();   // the backward: A comes from the launch before
  const int valid = min(T, max(__ldg(b.seg_ptr + b.S), 0));
  if (blockIdx.x < CTAS) {
    quantize_rows_cluster<CTAS>(x, valid, C, ld, out, CTAS == 1 ? 0 : cluster_ctarank());
    return;
  }
  __shared__ int row_id;
  __shared__ RowSums sums;
  const int item = blockIdx.x - CTAS, groups = b.rank / 8, t = item / groups, grp = item - t * groups;
  if (t >= T) return;
  const int found = row_adapter_of(b.seg_ptr, b.seg_adapter, b.S, b.count, t, &row_id), id = t < valid ? found : -2;
  if (grp == 0 && threadIdx.x == 0) row_adapter[t] = id;
  if (id < 0) return;
  row_low_rank(x + t * ld, A + (static_cast<int64_t>(id) * b.rank + grp * 8) * C, C, b.scale + id,
               V + static_cast<int64_t>(t) * b.rank + grp * 8, nullptr, sums);
}

struct RowsShape {
  int n_pad, stages, slices, keep;
  uint32_t tmem_cols, b_bytes, smem;
};

constexpr uint32_t kRing = 114432;

// Two CTAs an SM: each 114,432 bytes of ring at most (228 KB less what the
// kernel and the system keep) and 256 columns of tensor memory.  GATED with up
// to 16 rows of X takes half the columns, and with three stages a third of the
// memory: three CTAs an SM where that saves a wave (5120 by 2 x 28416, one row:
// 30 us, with two 41; 5120 by 2 x 18944, no wave less: 23.7 and 22.8).
RowsShape rows_shape(int T, int slices, int kind, int rank, bool three) {
  RowsShape s;
  s.n_pad = (T + 15) / 16 * 16;
  s.b_bytes = static_cast<uint32_t>(s.n_pad) * 128;
  s.slices = slices;
  s.keep = 0;
  if (kind == kAdapter) {
    const int mine = ((T + s.slices - 1) / s.slices + 3) / 4 * 4;
    s.keep = mine < KEEP ? mine : KEEP;
  }
  const uint32_t stage = A_BYTES + s.b_bytes + (kind == kGated ? 3 : 2) * SF_BYTES, kept = s.keep * (128 + rank) * 4;
  const int acc = (s.n_pad + 31) / 32 * 32, by_smem = static_cast<int>((kRing - kept) / stage), by_tmem = (256 - acc) / 32;
  s.stages = by_smem < by_tmem ? by_smem : by_tmem;
  if (s.stages > MAX_STAGES) s.stages = MAX_STAGES;
  if (three) s.stages = 3;
  const uint32_t cols = acc + s.stages * 32;
  s.tmem_cols = cols <= 128 ? 128 : 256;
  s.smem = s.stages * stage + kept + 1024;
  return s;
}

template <class Kernel>
cudaError_t launch_rows(Kernel kern, SmemOptIn* opt, const FpOperand& x, const FpOperand& w, int kind, int tiles,
                        RowsParams p, int num_sms, cudaStream_t s) {
  cudaError_t e = opt->ensure(kern, kRing + 1024);
  if (e != cudaSuccess) return e;
  const int n_pad = (p.T + 15) / 16 * 16, num_kt = (p.K + 255) / 256;
  CUtensorMap tmW, tmX;
  if (!operand_map(&tmW, w.data, p.N, p.K, kind == kGated ? 64 : 128) || !operand_map(&tmX, x.data, p.T, p.K, n_pad))
    return cudaErrorInvalidValue;
  p.sfw = w.scales;
  p.sfx = x.scales;
  p.gsw = w.gs;
  p.gsx = x.gs;
  auto launch = [&](int first, int count, int slices, bool three) {
    const RowsShape sh = rows_shape(p.T, slices, kind, p.rank, three);
    p.tile0 = first;
    p.n_pad = sh.n_pad;
    p.stages = sh.stages;
    p.slices = sh.slices;
    p.keep = sh.keep;
    p.tmem_cols = sh.tmem_cols;
    p.b_bytes = sh.b_bytes;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(count * sh.slices));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = sh.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(sh.slices);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tmW, tmX, p);
  };
  const int slots = 2 * num_sms, last = tiles % slots;   // two CTAs an SM
  if (kind == kGated && n_pad == 16 && (tiles + 3 * num_sms - 1) / (3 * num_sms) < (tiles + slots - 1) / slots)
    return launch(0, tiles, 1, true);
  // Whole waves first; then the tiles that are left, K split so that they, too,
  // use the whole GPU (5120 by 2 x 22528, 48 rows: 35 us, in one launch 43).
  const int tail = tiles > slots && last ? rows_slices(last, num_kt, num_sms) : 1;
  if (tail == 1) return launch(0, tiles, rows_slices(tiles, num_kt, num_sms), false);
  if ((e = launch(0, tiles - last, 1, false)) != cudaSuccess) return e;
  return launch(tiles - last, last, tail, false);
}

SmemOptIn g_opt_silu, g_opt_gelu, g_opt_adapter;

}  // namespace

cudaError_t read_rows_error(unsigned int* out, int clear) { return read_unit_error(out, clear); }

// CTAs of the quantizing cluster: one where a thread then has two blocks at
// most, eight where it has one, else sixteen (48 rows of 5120: 0.9 us less than
// eight; 64 rows 1.7 us less).
static int quant_ctas(int64_t T, int64_t C) {
  const int64_t blocks = T * (C / 16);
  return blocks <= 2 * kQuantThreads ? 1 : blocks <= 8 * kQuantThreads ? 8 : kMaxQuantCtas;
}

template <class Kernel, class... Args>
static cudaError_t launch_quant_cluster(Kernel kern, int ctas, int more, bool after, cudaStream_t s, Args... args) {
  if (ctas > 8) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas + (more + ctas - 1) / ctas * ctas));
  cfg.blockDim = dim3(kQuantThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_quant_few_rows(const void* x, int64_t T, int64_t C, int64_t ld, void* data, void* scales, float* gs,
                                  cudaStream_t s) {
  const QuantOut out{static_cast<uint8_t*>(data), static_cast<uint8_t*>(scales), gs, 0, 0, 0};
  auto* xs = static_cast<const uint16_t*>(x);
  const int t = static_cast<int>(T), c = static_cast<int>(C), ctas = quant_ctas(T, C);
  if (ctas == 1) return launch_quant_cluster(quant_few_rows_kernel<1>, 1, 0, false, s, xs, t, c, ld, out);
  if (ctas == 8) return launch_quant_cluster(quant_few_rows_kernel<8>, 8, 0, false, s, xs, t, c, ld, out);
  return launch_quant_cluster(quant_few_rows_kernel<kMaxQuantCtas>, kMaxQuantCtas, 0, false, s, xs, t, c, ld, out);
}

cudaError_t launch_lora_few_rows(const void* x, int64_t T, int64_t C, int64_t ld, int sr, uint64_t seed, void* data,
                                 void* scales, float* gs, const void* A, const LoraBatch& b, int* row_adapter, float* V,
                                 cudaStream_t s) {
  const QuantOut out{static_cast<uint8_t*>(data), static_cast<uint8_t*>(scales), gs, sr, static_cast<uint32_t>(seed),
                     static_cast<uint32_t>(seed >> 32)};
  auto* xs = static_cast<const uint16_t*>(x);
  auto* as = static_cast<const uint16_t*>(A);
  const int t = static_cast<int>(T), c = static_cast<int>(C), ctas = quant_ctas(T, C), items = t * (b.rank / 8);
  if (ctas == 1) return launch_quant_cluster(lora_few_rows_kernel<1>, 1, items, sr, s, xs, t, c, ld, out, as, b, row_adapter, V);
  if (ctas == 8) return launch_quant_cluster(lora_few_rows_kernel<8>, 8, items, sr, s, xs, t, c, ld, out, as, b, row_adapter, V);
  return launch_quant_cluster(lora_few_rows_kernel<kMaxQuantCtas>, kMaxQuantCtas, items, sr, s, xs, t, c, ld, out, as, b,
                              row_adapter, V);
}

cudaError_t launch_gated_rows(const FpOperand& x, const FpOperand& w, int64_t T, int64_t F, int64_t K, int act, void* H,
                              int64_t ldh, int num_sms, cudaStream_t s) {
  RowsParams p = {};
  p.T = static_cast<int>(T);
  p.N = static_cast<int>(2 * F);
  p.K = static_cast<int>(K);
  p.out = static_cast<__nv_bfloat16*>(H);
  p.ldo = ldh;
  const int tiles = static_cast<int>(F / 64);
  return act ? launch_rows(project_rows_kernel<kGated, 1>, &g_opt_gelu, x, w, kGated, tiles, p, num_sms, s)
             : launch_rows(project_rows_kernel<kGated, 0>, &g_opt_silu, x, w, kGated, tiles, p, num_sms, s);
}

cudaError_t launch_adapter_rows(const FpOperand& x, const FpOperand& w, int64_t T, int64_t N, int64_t K,
                                const int* row_adapter, const float* V, const void* B, int64_t rank, void* Y, int64_t ldy,
                                int num_sms, cudaStream_t s) {
  RowsParams p = {};
  p.T = static_cast<int>(T);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.out = static_cast<__nv_bfloat16*>(Y);
  p.ldo = ldy;
  p.V = V;
  p.row_adapter = row_adapter;
  p.B = static_cast<const __nv_bfloat16*>(B);
  p.rank = static_cast<int>(rank);
  return launch_rows(project_rows_kernel<kAdapter, 0>, &g_opt_adapter, x, w, kAdapter, static_cast<int>((N + 127) / 128),
                     p, num_sms, s);
}

}  // namespace nvfp4
