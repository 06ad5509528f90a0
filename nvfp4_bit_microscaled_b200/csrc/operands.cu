// operands.cu -- what a projection by tiles of 256 rows reads, from BF16 rows:
// the per-tensor amax, the row copy, and for low-rank adapters the slabs.
// Bound by memory: x is read twice (the second time from L2 where it fits) and
// written at 9/32 of its size.  1777 x 5120: amax and copy 11 us; 8192 x 8192:
// the copy and eight adapters' slabs 37 us after the amax (4.6 TB/s).
#include "tile.cuh"

namespace nvfp4 {

namespace {

// max |x| over rows with a pitch, one maximum (BF16 bits) for each block: the
// next launch takes the maximum of those (no memory has to be zeroed before).
__global__ void __launch_bounds__(256) rows_amax_kernel(const uint16_t* __restrict__ x, int64_t ldx, int64_t T, int C,
                                                        uint32_t* __restrict__ maxima) {
  __shared__ uint32_t warp_max[8];
  constexpr int U = 4;   // 16-byte loads in flight for each thread
  allow_next_kernel();
  const int64_t c8 = C / 8, items = T * c8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x, step_q = step / c8, step_r = step - step_q * c8;
  int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, r = i / c8, c = i - r * c8;
  uint32_t m = 0;
  while (i < items) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = i < items ? __ldg(reinterpret_cast<const uint4*>(x + r * ldx) + c) : make_uint4(0, 0, 0, 0);
      i += step;
      c += step_r;
      r += step_q;
      if (c >= c8) c -= c8, ++r;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m = max(m, absmax_bits8(v[u]));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 8) {
    m = __reduce_max_sync(0xFFu, warp_max[threadIdx.x]);
    if (threadIdx.x == 0) maxima[blockIdx.x] = m;
  }
}

// ---------------------------------------------------------------------------
// The operands of a projection by tiles, in one launch that needs the amax (and
// V).
//
// The first blocks quantize the valid rows of x (1x16 blocks, to nearest or
// stochastic): the arithmetic and the draws of quantize.cu's row kernel, warp
// item 32 blocks of a row, lane = block.
//
// Then slabs: for each adapter that a 256-row tile has rows of, V / alpha as two
// BF16 terms (the value rounded, and what that leaves, rounded: 16 bits of it, as
// one term's 8 would add half of the output's own rounding), zero in the other
// rows and past the rank.  [256][groups of 32 ranks][2 terms][32].  Up to rank 32
// the second term costs nothing (a step has room for both); rank 64, 2048 rows of
// 4096 x 4096 with 32 adapters 54 us with one term and 59 with two, 8192 rows of
// 8192 x 8192 with eight 276 and 278.
// alpha = s_gX s_gW: the accumulator the slab is multiplied into is scaled by it
// at the end.  Eight blocks write a slab, 32 rows each.  Where a finite V / alpha
// or its products would leave FP32's range (alpha may be a subnormal, or zero),
// the tile is marked: its epilogue adds V's products itself, after alpha.
// ---------------------------------------------------------------------------
struct OperandParams {
  const uint16_t* x;
  int64_t ldx;
  int T, K;
  const int* valid_rows;   // or null: all T rows
  const float* amax;         // or null: the maximum of
  const uint32_t* maxima;    // BF16 bits
  int num_maxima;
  uint32_t k0, k1;
  uint8_t* data;
  uint8_t* sf;
  float* gs_out;
  int quant_blocks;
  // slabs
  const float* V;
  int rank, rank_pad, count, parts;   // rank_pad: a multiple of 32
  const int* tile_count;
  const int* tile_base;
  const int* slab_adapter;
  const int* row_adapter;
  int* tile_direct;
  const int* second_max;
  const float* gs_w;
  int* slab_source;
  __nv_bfloat16* slabs;
};

__device__ void slab_part(const OperandParams& p, int slab, int part, int* sh) {
  if (threadIdx.x == 0) sh[0] = -1;
  __syncthreads();
  for (int k = threadIdx.x; k < (p.T + 255) / 256; k += blockDim.x)
    if (slab >= p.tile_base[k] && slab < p.tile_base[k] + p.tile_count[k]) sh[0] = k;
  __syncthreads();
  const int tile = sh[0];
  if (tile < 0) return;
  const int id = p.slab_adapter[slab];
  if (threadIdx.x < 32) {
    const int m = threadIdx.x < p.parts ? p.second_max[id * kCheckParts + threadIdx.x] : 0;
    const int most = __reduce_max_sync(0xFFFFFFFFu, m);
    if (threadIdx.x == 0) sh[1] = most;
  }
  __syncthreads();
  // an adapter with a value that is not finite: NaN for its own rows, and an
  // index past the adapters, whose rows the tile's loads fill with zeros
  const bool bad = sh[1] >= 0x7F80;
  if (part == 0 && threadIdx.x == 0) p.slab_source[slab] = bad ? p.count : id;
  const float alpha = __fmul_rn(decode_scale(*p.amax), __ldg(p.gs_w)), inv = __fdiv_rn(1.0f, alpha);
  const float second = bf16_bits_to_f32(sh[1]);
  bool over = false;
  // up to 128 products and the FP4 sum (below 2^48) stay below 2^104
  auto leaves = [&](float v, float z) { return isfinite(v) && !(fabsf(z) < 0x1p127f && fabsf(z) * second < 0x1p96f); };
  const int words = p.rank_pad / 8;
  for (int u = threadIdx.x; u < 32 * words; u += blockDim.x) {
    const int row = 32 * part + u / words, j = u % words * 8, t = tile * 256 + row;
    const bool own = t < p.T && p.row_adapter[t] == id;
    __nv_bfloat162 hi[4], lo[4];
    if (own && bad) {
      *reinterpret_cast<uint4*>(hi) = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
      *reinterpret_cast<uint4*>(lo) = make_uint4(0, 0, 0, 0);
    } else if (own && j < p.rank) {
      const float4* v = reinterpret_cast<const float4*>(p.V + static_cast<int64_t>(t) * p.rank + j);
      const float4 a = v[0], b = v[1];
      const float2 z[4] = {make_float2(a.x * inv, a.y * inv), make_float2(a.z * inv, a.w * inv),
                           make_float2(b.x * inv, b.y * inv), make_float2(b.z * inv, b.w * inv)};
      const float2 from[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        split_bf16x2(z[k], &hi[k], &lo[k]);
        over = over || leaves(from[k].x, z[k].x) || leaves(from[k].y, z[k].y);
      }
    } else {
      *reinterpret_cast<uint4*>(hi) = *reinterpret_cast<uint4*>(lo) = make_uint4(0, 0, 0, 0);
    }
    __nv_bfloat16* to = p.slabs + ((static_cast<int64_t>(slab) * 256 + row) * p.rank_pad + (j & ~31)) * 2 + (j & 31);
    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<uint4*>(hi);
    *reinterpret_cast<uint4*>(to + 32) = *reinterpret_cast<uint4*>(lo);
  }
  // (a scale that is not finite flags the whole batch: NaN whatever is added)
  if (__syncthreads_or(over && isfinite(alpha)) && threadIdx.x == 0) p.tile_direct[tile] = 1;
}

// NARROW: every block counter (element index / 16) fits in 32 bits.
template <bool SR, bool NARROW>
__device__ __forceinline__ void quantize_valid_rows(const OperandParams& p, float* r_tbl) {
  constexpr int U = SR ? 1 : 2;   // items in flight for each warp
  float amax;
  if (p.amax) {
    amax = *p.amax;
  } else {
    __shared__ uint32_t warp_max[8];
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.num_maxima; i += blockDim.x) m = max(m, p.maxima[i]);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
    amax = bf16_bits_to_f32(m);
  }
  const float s_enc = encode_scale(amax);
  const bool flagged = !isfinite(amax);   // as quantize.cu: NaN scales, zero codes
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.gs_out = decode_scale(amax);
  fill_r_table(r_tbl, s_enc);
  __syncthreads();
  const int lane = threadIdx.x & 31, S = p.K / 16, nseg = (S + 31) / 32;
  const int rows = p.valid_rows ? min(p.T, *p.valid_rows) : p.T;
  const int64_t items = static_cast<int64_t>(rows) * nseg, half = p.K / 2;
  const int64_t nwarps = static_cast<int64_t>(p.quant_blocks) * (blockDim.x >> 5);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); base < items;
       base += U * nwarps) {
    uint4 v[U][2];
    int64_t row[U];
    int blk[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t it = base + u * nwarps;
      row[u] = it / nseg;
      blk[u] = static_cast<int>(it - row[u] * nseg) * 32 + lane;
      ok[u] = it < items && blk[u] < S;
      v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (ok[u]) {
        const uint4* src = reinterpret_cast<const uint4*>(p.x + row[u] * p.ldx + blk[u] * 16);
        v[u][0] = __ldcs(src);
        v[u][1] = __ldcs(src + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * nwarps >= items) break;   // warp-uniform
      const uint4 a = v[u][0], b = v[u][1];
      const float2 y[8] = {bf16x2_to_f32x2(a.x), bf16x2_to_f32x2(a.y), bf16x2_to_f32x2(a.z), bf16x2_to_f32x2(a.w),
                           bf16x2_to_f32x2(b.x), bf16x2_to_f32x2(b.y), bf16x2_to_f32x2(b.z), bf16x2_to_f32x2(b.w)};
      BlockScale bs{0x7Fu, 0.0f};
      uint32_t w0 = 0, w1 = 0;
      if (!flagged) {
        bs = block_scale_t(bf16_bits_to_f32(max(absmax_bits8(a), absmax_bits8(b))), s_enc, r_tbl);
        const float2 r2 = make_float2(bs.r, bs.r);
        float2 z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = __fmul2_rn(y[k], r2);
        if (SR) {
          const u32x4 w = sr_words<NARROW>(static_cast<uint64_t>(row[u]) * S + blk[u], kDomainRowSR, p.k0, p.k1);
          w0 = sr_e2m1x4(z[0].x, z[0].y, z[1].x, z[1].y, w.x) | (sr_e2m1x4(z[2].x, z[2].y, z[3].x, z[3].y, w.y) << 16);
          w1 = sr_e2m1x4(z[4].x, z[4].y, z[5].x, z[5].y, w.z) | (sr_e2m1x4(z[6].x, z[6].y, z[7].x, z[7].y, w.w) << 16);
        } else {
          w0 = f32x8_to_e2m1x8(z[0].x, z[0].y, z[1].x, z[1].y, z[2].x, z[2].y, z[3].x, z[3].y);
          w1 = f32x8_to_e2m1x8(z[4].x, z[4].y, z[5].x, z[5].y, z[6].x, z[6].y, z[7].x, z[7].y);
        }
        w0 = clear_negative_zero(w0);
        w1 = clear_negative_zero(w1);
      }
      if (ok[u]) *reinterpret_cast<uint2*>(p.data + row[u] * half + blk[u] * 8) = make_uint2(w0, w1);
      uint32_t word = ok[u] ? bs.sf << (8 * (lane & 3)) : 0u;
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
      if ((lane & 3) == 0 && ok[u]) *reinterpret_cast<uint32_t*>(p.sf + sf_offset(row[u], blk[u], S)) = word;
    }
  }
}

template <bool SR, bool NARROW>
__global__ void __launch_bounds__(256, 4) tile_operands_kernel(const __grid_constant__ OperandParams p) {
  __shared__ float r_tbl[kRTableSize];
  __shared__ int sh[2];
  allow_next_kernel();
  wait_previous_kernel();
  if (blockIdx.x < static_cast<unsigned>(p.quant_blocks)) {
    quantize_valid_rows<SR, NARROW>(p, r_tbl);
  } else {
    const int u = blockIdx.x - p.quant_blocks;
    slab_part(p, u >> 3, u & 7, sh);
  }
}

OperandParams rows_params(const void* x, int64_t ldx, int64_t T, int64_t K, const int* valid_rows, const float* amax,
                          uint64_t seed, void* data, void* scales, float* gs, int num_sms) {
  OperandParams q = {};
  q.x = static_cast<const uint16_t*>(x);
  q.ldx = ldx;
  q.T = static_cast<int>(T);
  q.K = static_cast<int>(K);
  q.valid_rows = valid_rows;
  q.amax = amax;
  q.k0 = static_cast<uint32_t>(seed);
  q.k1 = static_cast<uint32_t>(seed >> 32);
  q.data = static_cast<uint8_t*>(data);
  q.sf = static_cast<uint8_t*>(scales);
  q.gs_out = gs;
  // one resident wave of four CTAs an SM (16 for each SM: 2 us more of 288, 64: 8)
  const int64_t blocks = (T * ((K / 16 + 31) / 32) + 15) / 16, cap = 4LL * num_sms;
  q.quant_blocks = static_cast<int>(blocks < cap ? blocks : cap);
  return q;
}

cudaError_t run_operands(const OperandParams& q, int sr, unsigned grid, cudaStream_t s) {
  if (!sr) return launch_after(tile_operands_kernel<false, false>, grid, 256, 0, s, q);
  return static_cast<int64_t>(q.T) * q.K < (int64_t(1) << 36)
             ? launch_after(tile_operands_kernel<true, true>, grid, 256, 0, s, q)
             : launch_after(tile_operands_kernel<true, false>, grid, 256, 0, s, q);
}

}  // namespace

cudaError_t launch_rows_operand(const void* x, int64_t ldx, int64_t T, int64_t K, void* maxima, void* data, void* scales,
                                float* gs, int num_sms, cudaStream_t s) {
  const int64_t blocks = (T * (K / 8) + 1023) / 1024, cap = 8LL * num_sms < kRowMaxima ? 8LL * num_sms : kRowMaxima;
  const int grid = static_cast<int>(blocks < cap ? blocks : cap);
  rows_amax_kernel<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(x), ldx, T, static_cast<int>(K),
                                        static_cast<uint32_t*>(maxima));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  OperandParams q = rows_params(x, ldx, T, K, nullptr, nullptr, 0, data, scales, gs, num_sms);
  q.maxima = static_cast<const uint32_t*>(maxima);
  q.num_maxima = grid;
  return run_operands(q, 0, static_cast<unsigned>(q.quant_blocks), s);
}

cudaError_t launch_lora_operands(const void* x, int64_t ldx, int64_t T, int64_t K, int sr, uint64_t seed, void* data,
                                 void* scales, float* gs, const float* V, int64_t N, const LoraBatch& b, const LoraPlan& p,
                                 const float* gs_w, bool slabs, int num_sms, cudaStream_t s) {
  OperandParams q = rows_params(x, ldx, T, K, p.valid_rows, p.amax, seed, data, scales, gs, num_sms);
  q.V = V;
  q.rank = b.rank;
  q.rank_pad = (b.rank + 31) / 32 * 32;
  q.count = b.count;
  q.parts = check_parts(N * b.rank);
  q.tile_count = p.tile_count;
  q.tile_base = p.tile_base;
  q.slab_adapter = p.slab_adapter;
  q.row_adapter = p.row_adapter;
  q.tile_direct = p.tile_direct;
  q.second_max = p.second_max;
  q.gs_w = gs_w;
  q.slab_source = p.slab_source;
  q.slabs = static_cast<__nv_bfloat16*>(p.slabs);
  const unsigned grid = static_cast<unsigned>(q.quant_blocks + (slabs ? 8 * (b.S + (T + 255) / 256) : 0));
  return run_operands(q, sr, grid, s);
}

}  // namespace nvfp4
