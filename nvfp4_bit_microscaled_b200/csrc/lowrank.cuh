// lowrank.cuh -- V = scale_i x A_i^T for one row of x and eight ranks, by one
// block: the form for rows whose requests are too short for a tile.
#pragma once
#include "tile.cuh"

namespace nvfp4 {

constexpr int kRowThreads = 512;   // at most

struct RowSums {
  float v[kRowThreads / 32][8];
  uint32_t m[kRowThreads / 32];
};

// The block's warps split the C columns; v[0 .. 7] = scale * sum_c x[c] a[j][c],
// summed in warp order.  a == nullptr: no product.  amax != nullptr: max |x|
// too.  a may come from a launch that this one overlaps.  Waits for the launch before (see wait_previous_kernel).  Block-wide.
__device__ __forceinline__ void row_low_rank(const uint16_t* __restrict__ x, const uint16_t* a, int C,
                                             const float* __restrict__ scale, float* __restrict__ v,
                                             unsigned int* __restrict__ amax, RowSums& sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float acc[8] = {};
  uint32_t m = 0;
  for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
    const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x + c));
    if (amax) m = max(m, absmax_bits8(xv));
    if (!a) continue;
    uint4 av[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) av[j] = *reinterpret_cast<const uint4*>(a + static_cast<int64_t>(j) * C + c);
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t aw[4] = {av[j].x, av[j].y, av[j].z, av[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 p = bf16x2_to_f32x2(xw[k]), q = bf16x2_to_f32x2(aw[k]);
        acc[j] = __fmaf_rn(p.y, q.y, __fmaf_rn(p.x, q.x, acc[j]));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
  if (amax) m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sums.v[warp][j] = acc[j];
    sums.m[warp] = m;
  }
  __syncthreads();
  if (a && threadIdx.x < 8) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w)
      if (w < static_cast<int>(blockDim.x >> 5)) s += sums.v[w][threadIdx.x];
    v[threadIdx.x] = s * __ldg(scale);
  }
  wait_previous_kernel();   // *amax is zero
  if (amax && threadIdx.x < 32) {
    m = __reduce_max_sync(0xFFFFFFFFu, threadIdx.x < blockDim.x / 32 ? sums.m[threadIdx.x] : 0u);
    if (threadIdx.x == 0 && m) atomicMax(amax, m << 16);
  }
}

// The adapter of row t: of the request that has it, -1 for none.  Three
// independent loads for each request, then the comparison.  Block-wide.
__device__ __forceinline__ int row_adapter_of(const int* __restrict__ seg_ptr, const int* __restrict__ seg_adapter, int S,
                                              int count, int t, int* found) {
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    const int lo = __ldg(seg_ptr + s), hi = __ldg(seg_ptr + s + 1), id = __ldg(seg_adapter + s);
    if (t >= lo && t < hi && id >= 0 && id < count) *found = id;
  }
  __syncthreads();
  return *found;
}

}  // namespace nvfp4
