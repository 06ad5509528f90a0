// tile.cuh -- host and device parts shared by the projection kernels
// (project.cu: tiles of many rows; rows.cu: few rows): tensor-map encoding,
// per-device kernel setup, the BF16 tensor-core instruction and the gate
// of the forward.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {

// --------------------------------------------------------------------------
// Host: tensor maps and launch setup
// --------------------------------------------------------------------------
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D map of [dim1, dim0] elements (dim0 contiguous, row pitch in bytes), box
// box1 x box0, 128-byte swizzle: one box row is exactly 128 bytes wide.
inline bool encode_map(CUtensorMap* tm, CUtensorMapDataType type, const void* base, int64_t dim0, int64_t dim1,
                       int64_t pitch_bytes, int box0, int box1, CUtensorMapL2promotion l2) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(dim0), static_cast<cuuint64_t>(dim1)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box0), static_cast<cuuint32_t>(box1)};
  cuuint32_t estr[2] = {1, 1};
  return encode(tm, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed FP4 operand [rows, K / 2] bytes, boxes of 128 bytes x box_rows.
inline bool operand_map(CUtensorMap* tm, const void* data, int64_t rows, int64_t K, int box_rows) {
  return encode_map(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, data, K / 2, rows, K / 2, 128, box_rows,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// BF16 matrix [rows, cols] with row pitch ld (elements), boxes of 64 columns x
// box_rows.  loads: L2 fetches 256 bytes, the next box of the row with this one.
inline bool bf16_map(CUtensorMap* tm, const void* data, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                     bool loads = false) {
  return encode_map(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, data, cols, rows, ld * 2, 64, box_rows,
                    loads ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// Dynamic shared-memory opt-in, once per device and kernel.
struct SmemOptIn {
  std::mutex mu;
  bool done[64] = {};
  template <class Kernel>
  cudaError_t ensure(Kernel kern, uint32_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    done[dev] = e == cudaSuccess;
    return e;
  }
};

#ifdef NVFP4_UNIT_ERROR_WORD
// The including unit's own error word (synchronous); clear != 0 resets it.
inline cudaError_t read_unit_error(unsigned int* out, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_device_error, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(unsigned int));
}
#endif

#ifdef __CUDACC__
// A launch that may begin beside the end of the one before it (the kernel waits
// for that one itself before it touches memory).
template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kern, unsigned grid, unsigned threads, uint32_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// --------------------------------------------------------------------------
// Device
// --------------------------------------------------------------------------
// Programmatic dependent launch: a kernel launched so may start once the one
// before it allows it, and waits for that one's end (and its memory) here.  What
// a launch of the same call writes is read by ordinary loads after the wait, not
// through the read-only path (__ldg, const __restrict__ parameters): that is for
// data that stays as it is while the kernel lives, which begins before the wait.
__device__ __forceinline__ void wait_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Pair MMA on BF16 operands, K = 16, FP32 accumulation (leader CTA only).
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same on one CTA (M = 128).
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two FP32 values as a BF16 term and the BF16 rounding of what it leaves (an
// infinity leaves nothing).
__device__ __forceinline__ void split_bf16x2(float2 v, __nv_bfloat162* hi, __nv_bfloat162* lo) {
  *hi = __floats2bfloat162_rn(v.x, v.y);
  const float2 h = __bfloat1622float2(*hi);
  *lo = __floats2bfloat162_rn(fabsf(h.x) == INFINITY ? 0.0f : v.x - h.x, fabsf(h.y) == INFINITY ? 0.0f : v.y - h.y);
}

template <int N>
__device__ __forceinline__ void regs_release() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_claim() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// s = sigmoid(q(g)) with act(g) = g s: q(g) = g (SiLU) or, for the tanh form
// of GELU, q(g) = 2 sqrt(2/pi) (g + 0.044715 g^3), as (1 + tanh z) / 2 =
// sigmoid(2 z).  Beyond |g| = 30 both are 0 or 1 in FP32; the clamp keeps g^3
// finite.  The fast exponential's error grows with its argument, about |q| ulps,
// and reaches the 90 or so where the sigmoid still differs from 0 or 1; the fast
// division adds two.  128 ulps are a 512th of the rounding of H to BF16.
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;
template <int ACT>
__device__ __forceinline__ float gate_sigmoid(float g) {
  if (ACT == 1) {
    const float c = fminf(fmaxf(g, -30.0f), 30.0f);
    g = kGeluA * __fmaf_rn(kGeluB * c * c, c, c);
  }
  return __fdividef(1.0f, 1.0f + __expf(-g));
}
#endif

}  // namespace nvfp4
