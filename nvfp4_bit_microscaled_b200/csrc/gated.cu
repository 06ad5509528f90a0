// gated.cu -- backward of the gated projection, up to the GEMMs: the gradient
// of G | U, quantized for dgrad (row copy) and wgrad (transposed copy with the
// RHT), both with stochastic rounding.
//
//   H = act(G) U:  dG = dH U act'(G),  dU = dH act(G)
//
// dG | dU [T, 2F] is never stored.  Two kernels read dH, G and U (6 bytes for
// two gradients): one takes the two maxima, one makes both copies.  Each
// computes the products in FP32, and nothing is rounded before the quantizer's
// own rounding.  Storing the gradients as BF16 would cost 8 bytes for the pair
// (written, read twice) on top of the same reads once.
// The exponential and the hyperbolic tangent are CUDA's accurate ones, and the
// sigmoid's reciprocal is the hardware's approximation after one Newton step
// (within an ulp or two): a gradient that is off in its last bits can change a
// random draw's outcome, and with it a code by a whole step.
// Measured (8192 tokens, F = 10240, SiLU; 503 MB of input): the maxima 138 us
// (3.6 TB/s), the copies 306 us.  Both are bound by instructions: 38 for a pair
// of gradients in the first kernel, issue slots 57-67% busy, DRAM 19-38%.  Input
// tiles that TMA brings ahead of time changed neither (137 and 330 us), nor did
// twice the warps with half the channels each (141 and 350 us).
#include "tile.cuh"

namespace nvfp4 {

namespace {

// act(g) and act'(g) (SiLU; GELU in its tanh form).  Beyond |g| = 30 the tanh
// form's gate is 0 or 1; the clamp keeps its powers of g finite.
template <int ACT>
__device__ __forceinline__ void gate(float g, float* a, float* da) {
  if (ACT == 0) {
    // the reciprocal of x = 1 + e^-g by one Newton step (r + r (1 - x r), with
    // fused steps: Markstein, IBM J. Res. Dev. 34(1), 1990) on the hardware's
    // approximation.  Where x is infinite r is 0, and the bound keeps x r from
    // 0 x infinity: s is 0.
    const float x = 1.0f + expf(-g);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    const float s = __fmaf_rn(r, __fmaf_rn(-fminf(x, 1e38f), r, 1.0f), r);
    *a = g * s;
    *da = s * (1.0f + g * (1.0f - s));
  } else {
    const float k = 0.7978845608028654f, c = 0.044715f, x = fminf(fmaxf(g, -30.0f), 30.0f);
    const float t = tanhf(k * (x + c * x * x * x));
    *a = 0.5f * g * (1.0f + t);
    *da = 0.5f * (1.0f + t) + 0.5f * x * (1.0f - t * t) * k * (1.0f + 3.0f * c * x * x);
  }
}

// dG and dU of two neighbouring channels (packed BF16 words).
template <int ACT>
__device__ __forceinline__ void gate_pair_x2(uint32_t dh, uint32_t g, uint32_t u, float2* dg, float2* du) {
  const float2 h2 = bf16x2_to_f32x2(dh), g2 = bf16x2_to_f32x2(g), u2 = bf16x2_to_f32x2(u);
  float2 a, d;
  gate<ACT>(g2.x, &a.x, &d.x);
  gate<ACT>(g2.y, &a.y, &d.y);
  *dg = __fmul2_rn(__fmul2_rn(h2, u2), d);
  *du = __fmul2_rn(h2, a);
}

// Tiles of 64 tokens x 128 channels of dH, G and U.  A warp takes 16 tokens
// (its band) x 64 channels, a thread two channels: 128 contiguous bytes of a
// row for each load, and the 16-token blocks of both channels in registers.
// Offsets inside a tile are 32-bit (15 rows).
constexpr int kTileTokens = 64, kTileChannels = 128;

struct TileAt {
  const uint16_t* h;   // this thread's first token and channel of dH
  const uint16_t* g;   // of G; U is F elements on
};
__device__ __forceinline__ TileAt tile_at(const uint16_t* dh, const uint16_t* gu, int64_t F, int64_t q, int64_t cb, int warp,
                                          int lane) {
  const int64_t t = q * kTileTokens + 16 * (warp >> 1), c = cb * kTileChannels + 64 * (warp & 1) + 2 * lane;
  return TileAt{dh + t * F + c, gu + t * 2 * F + c};
}

// The gradients of the thread's 16 tokens x 2 channels: v[0] dG, v[1] dU.
template <int ACT>
__device__ __forceinline__ void load_gradients(const TileAt& at, uint32_t F, float2 (&v)[2][16]) {
  uint32_t h[16], g[16], u[16];
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) {
    h[i] = __ldcs(reinterpret_cast<const unsigned int*>(at.h + i * F));
    g[i] = __ldcs(reinterpret_cast<const unsigned int*>(at.g + i * 2 * F));
    u[i] = __ldcs(reinterpret_cast<const unsigned int*>(at.g + (i * 2 * F + F)));
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) gate_pair_x2<ACT>(h[i], g[i], u[i], &v[0][i], &v[1][i]);
}

// max |dG|, |dU| (out[0]) and the maximum after the RHT along tokens (out[1]).
// A maximum drops NaN, so every gradient times zero is added to a sum that
// stays zero unless one was not finite; then both results are NaN (its bit
// pattern orders above every number's).
template <int ACT>
__global__ void __launch_bounds__(256, 2) gated_grad_amax_kernel(const uint16_t* __restrict__ dh,
                                                                 const uint16_t* __restrict__ gu, int64_t T, int64_t F,
                                                                 unsigned int* __restrict__ out) {
  float m = 0.0f, plain = 0.0f;
  float2 poison = make_float2(0.0f, 0.0f);
  const float2 zero = make_float2(0.0f, 0.0f);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t nc = F / kTileChannels, tiles = (T / kTileTokens) * nc;
  allow_next_kernel();
  for (int64_t ti = blockIdx.x; ti < tiles; ti += gridDim.x) {
    const int64_t q = ti / nc;
    float2 v[2][16];
    load_gradients<ACT>(tile_at(dh, gu, F, q, ti - q * nc, warp, lane), static_cast<uint32_t>(F), v);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        plain = max3_abs(plain, v[p][i].x, v[p][i].y);
        poison = __ffma2_rn(v[p][i], zero, poison);
      }
      bool neg[16];
      fwht16_x2<3>(v[p], neg);
#pragma unroll
      for (int j = 0; j < 8; ++j)   // the last stage folds into the maximum: max |a +- b| = |a| + |b|
        m = max3f(m, __fadd_rn(fabsf(v[p][j].x), fabsf(v[p][j + 8].x)), __fadd_rn(fabsf(v[p][j].y), fabsf(v[p][j + 8].y)));
    }
  }
  const bool bad = poison.x != 0.0f || poison.y != 0.0f;   // NaN compares unequal
  uint32_t pb = bad ? 0x7FC00000u : __float_as_uint(plain);
  uint32_t rot = bad ? 0x7FC00000u : __float_as_uint(__fmul_rn(m, 0.25f));
  pb = __reduce_max_sync(0xFFFFFFFFu, pb);
  rot = __reduce_max_sync(0xFFFFFFFFu, rot);
  wait_previous_kernel();   // out is zero
  if (lane == 0) {
    if (pb) atomicMax(out, pb);
    if (rot) atomicMax(out + 1, rot);
  }
}

// A copy whose amax is not finite: NaN scales, zero codes (as quantize.cu does).
__device__ __noinline__ void flag_grad_copy(uint8_t* data, int64_t rows, int64_t row_bytes, uint8_t* sf, int64_t S) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t nt = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = t0; i < rows * row_bytes; i += nt) data[i] = 0;
  for (int64_t i = t0; i < rows * S; i += nt) sf[sf_offset(i / S, i % S, S)] = 0x7F;
}

// Both copies from one read.  The blocks in registers make the transposed copy:
// a thread has four blocks (two channels of dG and of dU), whose codes meet the
// other bands' in shared memory, so that a channel's 64 tokens leave as 32
// bytes and one scale word.  The gradients also go to shared memory, from which
// eight neighbouring threads read a token's eight 16-channel blocks for the row
// copy.  Shared memory, for dG and dU each: [64 tokens][8 blocks][4 chunks of 16
// bytes]; chunk k of block b sits in slot 4 b + (k ^ (b / 2 % 4)), so that eight
// threads that read chunk k of eight blocks hit distinct banks.
constexpr uint32_t kGradTileBytes = kTileTokens * kTileChannels * 4;
constexpr uint32_t kCodeBytes = 2 * kTileChannels * 32, kScaleBytes = 2 * kTileChannels * 4;

__device__ __forceinline__ uint32_t grad_slot(int token, int block, int chunk) {
  return static_cast<uint32_t>(token * (kTileChannels * 4) + ((4 * block + (chunk ^ ((block >> 1) & 3))) << 4));
}

template <int ACT>
__global__ void __launch_bounds__(256, 2) gated_grad_quant_kernel(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu, int64_t T, int64_t F, const float* amax_dev,
    uint32_t k0, uint32_t k1, uint8_t* __restrict__ row_data, uint8_t* __restrict__ row_sf, float* __restrict__ row_gs,
    uint8_t* __restrict__ col_data, uint8_t* __restrict__ col_sf, float* __restrict__ col_gs) {
  extern __shared__ __align__(16) uint8_t tile[];   // dG, dU, then the transposed copy's codes and scales
  uint8_t* codes = tile + 2 * kGradTileBytes;
  uint8_t* scales = codes + kCodeBytes;
  __shared__ float r_row[kRTableSize], r_col[kRTableSize];
  wait_previous_kernel();   // for the maxima
  const float a_row = amax_dev[0], a_col = amax_dev[1];
  const float se_row = encode_scale(a_row), se_col = encode_scale(a_col);
  const int64_t row_s = F >> 3, col_s = T >> 4;   // blocks of a row of each copy
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *row_gs = decode_scale(a_row);
    *col_gs = decode_scale(a_col);
  }
  const bool flag_row = !isfinite(a_row), flag_col = !isfinite(a_col);
  if (flag_row) flag_grad_copy(row_data, T, F, row_sf, row_s);
  if (flag_col) flag_grad_copy(col_data, 2 * F, T >> 1, col_sf, col_s);
  fill_r_table(r_row, se_row);
  fill_r_table(r_col, se_col);
  __syncthreads();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, band = warp >> 1;
  const int64_t nc = F / kTileChannels, tiles = (T / kTileTokens) * nc;
  for (int64_t ti = blockIdx.x; ti < tiles; ti += gridDim.x) {
    const int64_t q = ti / nc, cb = ti - q * nc;
    {
      float2 v[2][16];
      load_gradients<ACT>(tile_at(dh, gu, F, q, cb, warp, lane), static_cast<uint32_t>(F), v);
      const int ch = 64 * (warp & 1) + 2 * lane;   // channel in the tile
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t at = p * kGradTileBytes + grad_slot(16 * band, ch >> 4, (ch >> 2) & 3) + 8 * (lane & 1);
#pragma unroll
        for (int i = 0; i < 16; ++i) *reinterpret_cast<float2*>(tile + at + i * (kTileChannels * 4)) = v[p][i];
        if (flag_col) continue;
        bool neg[16];
        fwht16_x2(v[p], neg);
        const float m0 = __fmul_rn(absmax16<false>(v[p]), 0.25f), m1 = __fmul_rn(absmax16<true>(v[p]), 0.25f);
        const BlockScale b0 = block_scale_t(m0, se_col, r_col), b1 = block_scale_t(m1, se_col, r_col);
        // (v / 4) r = v (r / 4) bit for bit, as a quarter is exact; the true sign comes with it
        const float2 rp = make_float2(0.25f * b0.r, 0.25f * b1.r), rn = make_float2(-rp.x, -rp.y);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[p][i] = __fmul2_rn(v[p][i], neg[i] ? rn : rp);
        const uint64_t gb = static_cast<uint64_t>(4 * q + band) * (2 * F) +
                            static_cast<uint64_t>(p * F + cb * kTileChannels + ch);
        uint8_t* dst = codes + (p * kTileChannels + ch) * 32 + 8 * band;
        scales[(p * kTileChannels + ch) * 4 + band] = static_cast<uint8_t>(b0.sf);
        scales[(p * kTileChannels + ch) * 4 + 4 + band] = static_cast<uint8_t>(b1.sf);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          auto e = [&](int i) { return c ? v[p][i].y : v[p][i].x; };
          const u32x4 w = sr_words<true>(gb + c, kDomainColSR, k0, k1);
          *reinterpret_cast<uint2*>(dst + 32 * c) = make_uint2(
              clear_negative_zero(sr_e2m1x4(e(0), e(1), e(2), e(3), w.x) | (sr_e2m1x4(e(4), e(5), e(6), e(7), w.y) << 16)),
              clear_negative_zero(sr_e2m1x4(e(8), e(9), e(10), e(11), w.z) | (sr_e2m1x4(e(12), e(13), e(14), e(15), w.w) << 16)));
        }
      }
    }
    __syncthreads();
    if (!flag_col) {   // a thread for each of the tile's 2 x 128 channels
      const int64_t ch = (tid >> 7) * F + cb * kTileChannels + (tid & 127);
      uint4* dst = reinterpret_cast<uint4*>(col_data + ch * (T >> 1) + q * 32);
      dst[0] = reinterpret_cast<const uint4*>(codes + tid * 32)[0];
      dst[1] = reinterpret_cast<const uint4*>(codes + tid * 32)[1];
      *reinterpret_cast<uint32_t*>(col_sf + sf_offset(ch, 4 * q, col_s)) = reinterpret_cast<const uint32_t*>(scales)[tid];
    }
    if (!flag_row) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {   // dG tokens 0-31, 32-63, then dU
        const int p = k >> 1, token = 32 * (k & 1) + (tid >> 3), b = tid & 7;
        float2 y[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 f = *reinterpret_cast<const float4*>(tile + p * kGradTileBytes + grad_slot(token, b, c));
          y[2 * c] = make_float2(f.x, f.y);
          y[2 * c + 1] = make_float2(f.z, f.w);
        }
        float m = max3_abs(y[0].x, y[0].y, y[1].x);
#pragma unroll
        for (int i = 1; i < 7; ++i) m = max3_abs(m, y[i].y, y[i + 1].x);
        m = max3_abs(m, y[7].y, 0.0f);
        const BlockScale bs = block_scale_t(m, se_row, r_row);
        const float2 r2 = make_float2(bs.r, bs.r);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(y[i], r2);
        const int64_t t = q * 64 + token, blk = p * (F >> 4) + cb * 8 + b;
        const u32x4 w = sr_words<true>(static_cast<uint64_t>(t * row_s + blk), kDomainRowSR, k0, k1);
        *reinterpret_cast<uint2*>(row_data + t * F + blk * 8) = make_uint2(
            clear_negative_zero(sr_e2m1x4(y[0].x, y[0].y, y[1].x, y[1].y, w.x) |
                                (sr_e2m1x4(y[2].x, y[2].y, y[3].x, y[3].y, w.y) << 16)),
            clear_negative_zero(sr_e2m1x4(y[4].x, y[4].y, y[5].x, y[5].y, w.z) |
                                (sr_e2m1x4(y[6].x, y[6].y, y[7].x, y[7].y, w.w) << 16)));
        uint32_t word = bs.sf << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
        if ((lane & 3) == 0) {
          *reinterpret_cast<uint32_t*>(row_sf + sf_offset(t, blk, row_s)) = word;
          // T % 128 == 64: the last tokens' tile also zeroes the scale rows past the tensor
          if ((T & 64) && t + 64 >= T) *reinterpret_cast<uint32_t*>(row_sf + sf_offset(t + 64, blk, row_s)) = 0u;
        }
      }
    }
    __syncthreads();   // the tile is rewritten
  }
  if (flag_row && (T & 64))
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + tid; i < 64 * row_s; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
      row_sf[sf_offset(T + i / row_s, i % row_s, row_s)] = 0;
}

}  // namespace

cudaError_t launch_gated_grad_amax(const void* dH, const void* GU, int64_t T, int64_t F, int act, float* amax_dev,
                                   int num_sms, cudaStream_t s) {
  cudaError_t e = launch_zero(amax_dev, 2, s);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (T / kTileTokens) * (F / kTileChannels);
  const unsigned grid = static_cast<unsigned>(tiles < 2LL * num_sms ? tiles : 2LL * num_sms);   // one resident wave
  auto* h = static_cast<const uint16_t*>(dH);
  auto* g = static_cast<const uint16_t*>(GU);
  auto* out = reinterpret_cast<unsigned int*>(amax_dev);
  return act ? launch_after(gated_grad_amax_kernel<1>, grid, 256, 0, s, h, g, T, F, out)
             : launch_after(gated_grad_amax_kernel<0>, grid, 256, 0, s, h, g, T, F, out);
}

cudaError_t launch_gated_grad_quant(const void* dH, const void* GU, int64_t T, int64_t F, int act, const float* amax,
                                    uint64_t seed, void* row_data, void* row_scales, float* row_gs, void* col_data,
                                    void* col_scales, float* col_gs, int num_sms, cudaStream_t s) {
  const int64_t tiles = (T / kTileTokens) * (F / kTileChannels), cap = 2LL * num_sms;
  const unsigned grid = static_cast<unsigned>(tiles < cap ? tiles : cap);
  const uint32_t smem = 2 * kGradTileBytes + kCodeBytes + kScaleBytes, k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
  auto run = [&](auto kern, SmemOptIn* opt) {
    cudaError_t e = opt->ensure(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, grid, 256, smem, s, static_cast<const uint16_t*>(dH), static_cast<const uint16_t*>(GU), T, F,
                        amax, k0, k1, static_cast<uint8_t*>(row_data), static_cast<uint8_t*>(row_scales), row_gs,
                        static_cast<uint8_t*>(col_data), static_cast<uint8_t*>(col_scales), col_gs);
  };
  static SmemOptIn opts[2];
  return act ? run(gated_grad_quant_kernel<1>, &opts[0]) : run(gated_grad_quant_kernel<0>, &opts[1]);
}

}  // namespace nvfp4
