// kernels.h -- internal launchers behind the C ABI (not part of the public header).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Zeroes n <= 32 words; the launch after it may begin beside it (launch_after in
// tile.cuh) and waits before it uses them.  A memory node in its place costs 4 us
// in a graph.
cudaError_t launch_zero(void* words, int n, cudaStream_t s);
// rht: 0 max|x|, 1 max|Q x| (signs kRhtSignMask), 2 both (amax_dev[0], [1]).
cudaError_t launch_amax(const void* x, int64_t R, int64_t C, int64_t ld, int rht, float* amax_dev, int num_sms,
                        cudaStream_t s);

// Row-wise 1x16 quantization: data [R, C/2], scales in the 128x4-tile layout
// with sp = pad4(C/16) scale columns.  idx0: element index of x[0][0] in the
// tensor whose row-major index keys the SR draws (0 for a whole tensor).
cudaError_t launch_quant_row(const void* x, int64_t R, int64_t C, int64_t ld, const float* amax_dev, int sr,
                             uint64_t seed, int64_t idx0, void* data, void* scales, float* gs_out, int num_sms,
                             cudaStream_t s);

// Column-wise 1x16 quantization along R, optional RHT and SR; transposed
// output data [C, R/2], scales with sp = pad4(R/16).
cudaError_t launch_quant_col(const void* x, int64_t R, int64_t C, int64_t ld, const float* amax_dev, int rht,
                             int sr, uint64_t seed, int64_t idx0, void* data, void* scales, float* gs_out,
                             int num_sms, cudaStream_t s);

// Row copy (data [R, C/2]) and column copy (data [C, R/2], RHT along R when
// rht != 0) from one read of x, round to nearest; the row copy is scaled by
// *amax_row, the column copy by *amax_col.
cudaError_t launch_quant_rowcol(const void* x, int64_t R, int64_t C, int64_t ld, const float* amax_row,
                                const float* amax_col, int rht, void* row_data, void* row_scales, float* row_gs,
                                void* col_data, void* col_scales, float* col_gs, int num_sms, cudaStream_t s);

// MXFP4 row-wise 1x32 quantization: data [R, C/2], UE8M0 scales in the 128x4
// tile layout with sp = pad4(C/32); writes 1.0 to *gs_out when given.
cudaError_t launch_mx_quant_row(const void* x, int64_t R, int64_t C, int64_t ld, void* data, void* scales,
                                float* gs_out, int num_sms, cudaStream_t s);

// 2D 16x16 quantization of W [N, K]: row copy [N, K/2] and/or column copy [K, N/2].
cudaError_t launch_quant_2d(const void* w, int64_t N, int64_t K, int64_t ld, const float* amax_dev,
                            void* row_data, void* row_scales, float* row_gs, void* col_data, void* col_scales,
                            float* col_gs, int num_sms, cudaStream_t s);

// Self-test: the block-scale divide-by-6 against the IEEE division on every
// non-negative finite float (synchronous, default stream).
cudaError_t selftest_div6(unsigned long long* bad_quotients, unsigned long long* bad_codes, int num_sms);

// Self-test: the stochastic-rounding conversion against its rule, every
// 16-bit draw of every lane for a spread of values (synchronous).
cudaError_t selftest_sr(unsigned long long* mismatches, unsigned long long* checked);

// Zero the padding of a scale matrix (rows >= R or scale columns >= S).
cudaError_t launch_sf_pad_zero(void* scales, int64_t R, int64_t S, cudaStream_t s);

// Block-scaled FP4 GEMM: D[M,N] = sgA * sgB * sum_k A[m,k] B[n,k].  mx != 0:
// MXFP4 operands (UE8M0 scale per 32 elements, sgA = sgB = 1 pointers still
// read); it always runs on the CTA-pair kernel.  amax_out (NVFP4 only): the
// launcher zeroes *amax_out and the epilogue writes max |D| of the stored
// values there.
cudaError_t launch_gemm(const void* a_data, const void* a_scales, const float* a_gs, const void* b_data,
                        const void* b_scales, const float* b_gs, int64_t M, int64_t N, int64_t K, void* D,
                        int out_bf16, int64_t ldd, int num_sms, cudaStream_t s, int mx = 0,
                        float* amax_out = nullptr);

// A packed FP4 operand of the projection kernels: codes, block scales, decode scale.
struct FpOperand {
  const uint8_t* data;
  const uint8_t* scales;
  const float* gs;
};

// Gated projection, tiles of 256 rows: H = act(G) * U with G | U = A W^T, W
// [2F, K] (gate rows first).  GU (optional) receives G | U, [M, 2F] contiguous;
// amax_out (optional) max |H|.  act: 0 SiLU, 1 GELU (tanh form).
cudaError_t launch_gated_tiles(const FpOperand& a, const FpOperand& w, int64_t M, int64_t F, int64_t K, int act, void* H,
                               int64_t ldh, void* GU, float* amax_out, int num_sms, cudaStream_t s);

// Gradient of the gated projection's G | U from dH [T, F] and GU [T, 2F] (BF16,
// contiguous): amax_dev[0] = max |dG|, |dU| and amax_dev[1] = the maximum after
// the RHT along tokens; then the row copy [T, 2F] (SR, amax[0]) and the
// transposed copy [2F, T] (RHT, SR, amax[1]).
cudaError_t launch_gated_grad_amax(const void* dH, const void* GU, int64_t T, int64_t F, int act, float* amax_dev,
                                   int num_sms, cudaStream_t s);
cudaError_t launch_gated_grad_quant(const void* dH, const void* GU, int64_t T, int64_t F, int act, const float* amax,
                                    uint64_t seed, void* row_data, void* row_scales, float* row_gs, void* col_data,
                                    void* col_scales, float* col_gs, int num_sms, cudaStream_t s);

// Low-rank adapters (lora.cu).  A batch: its requests' row ranges and adapters
// (device), the adapters' scales and rank.
struct LoraBatch {
  const int* seg_ptr;       // [S + 1]
  const int* seg_adapter;   // [S]; outside [0, count): none
  int S;
  const float* scale;       // [count]
  int count, rank;
};

// Few rows (T <= kFewRows): amax and row-wise quantization in one launch (no
// scale padding is written: rows >= T of the scale tiles stay as they are, and
// only outputs of rows that do not exist depend on them), and the projections.
// A projection starts beside the quantizer, so one of the two that quantize has
// to be the launch before it, and must not write W.
constexpr int64_t kFewRows = 128;
cudaError_t launch_quant_few_rows(const void* x, int64_t T, int64_t C, int64_t ld, void* data, void* scales, float* gs,
                                  cudaStream_t s);
// The same of the rows before seg_ptr[S] (the others are neither read nor
// written; sr: stochastic rounding), and beside it their V = scale_i x
// A_i^T (A [count, rank, C] BF16) and row_adapter (see launch_adapter_rows).
cudaError_t launch_lora_few_rows(const void* x, int64_t T, int64_t C, int64_t ld, int sr, uint64_t seed, void* data,
                                 void* scales, float* gs, const void* A, const LoraBatch& b, int* row_adapter, float* V,
                                 cudaStream_t s);
cudaError_t launch_gated_rows(const FpOperand& x, const FpOperand& w, int64_t T, int64_t F, int64_t K, int act, void* H,
                              int64_t ldh, int num_sms, cudaStream_t s);
// K is split over the cluster where that makes more of the GPU work: the CTAs of
// a tile minimise waves x (K steps of a CTA + 3), 3 steps (of 256 columns) being
// about what a CTA costs beside its loop.
inline int rows_slices(int64_t tiles, int64_t num_kt, int num_sms) {
  int slices = 1;
  int64_t best = -1;
  for (int ks = 1; ks <= 8 && ks <= num_kt; ks *= 2) {
    // two CTAs an SM; clusters of 4 and 8 leave some of them unused (284 and 264 of 296 are resident)
    const int64_t slots = 2 * num_sms * (ks <= 2 ? 100 : ks == 4 ? 95 : 89) / 100;
    const int64_t cost = ((tiles * ks + slots - 1) / slots) * ((num_kt + ks - 1) / ks + 3);
    if (best < 0 || cost < best) best = cost, slices = ks;
  }
  return slices;
}
// row_adapter [T]: the row's adapter, -1 none, -2 a padding row (left alone).
cudaError_t launch_adapter_rows(const FpOperand& x, const FpOperand& w, int64_t T, int64_t N, int64_t K,
                                const int* row_adapter, const float* V, const void* B, int64_t rank, void* Y, int64_t ldy,
                                int num_sms, cudaStream_t s);

// What the adapter tiles read besides the operands, made on the device by
// lora.cu: the rows in use, for each 256-row tile how many adapters' slabs it
// has (tile_count) and the first one's index (tile_base), each slab's adapter
// (`count`: none, zeros), and the slabs, [max_slabs][256][ranks / 32, rounded up]
// [2 terms][32] BF16.
struct AdapterPlan {
  const int* valid_rows;
  const int* tile_count;
  const int* tile_base;
  const int* slab_adapter;
  const void* slabs;
  int64_t max_slabs;
  // Tiles whose slabs cannot hold V / alpha (tile_direct not 0) take V [T, rank]
  // FP32 itself, by each row's adapter (-1 or -2: none).
  const int* tile_direct;
  const float* V;
  const int* row_adapter;
};

// Y = A W^T + (slabs) (adapter rows)^T, tiles of 256 rows; adapter_rows
// [adapters * N, rank] BF16.  Rows from *plan.valid_rows on are left alone.
cudaError_t launch_adapter_tiles(const FpOperand& a, const FpOperand& w, int64_t M, int64_t N, int64_t K,
                                 const AdapterPlan& plan, const void* adapter_rows, int64_t adapters, int64_t rank,
                                 void* Y, int64_t ldy, int num_sms, cudaStream_t s);

// Workspace parts that the shrink launch fills for the kernels after it.
struct LoraPlan {
  int* valid_rows;     // seg_ptr[S], clamped to the batch
  int* tile_count;     // per 256-row tile: slabs
  int* tile_base;      // per 256-row tile: first slab
  int* slab_adapter;   // per slab: its adapter
  int* slab_source;    // the same, `count` where the adapter is kept out (written with the slabs)
  int* row_adapter;    // per row: adapter, -1 none, -2 padding
  int* tile_direct;    // per 256-row tile: low-rank products in the epilogue (written with the slabs)
  int* second_max;     // per adapter, 32 parts: largest magnitude of the second operand, BF16 bits
  void* slabs;
  float* amax;         // max |x| over the requests' rows
};

// V[t, :] = scale_i x[t, :] A_i^T (A [count, rank, K] BF16) for rows of requests
// with an adapter, the plan, and *p.amax (zeroed: it is 0 already).  E: NULL, or
// the second operands ([count, N, rank]) of slabs to come, whose maxima are taken.
cudaError_t launch_lora_shrink(const void* x, int64_t ldx, int64_t T, int64_t K, const void* A, const void* E, int64_t N,
                               const LoraBatch& b, const LoraPlan& p, bool zeroed, float* V, int num_sms,
                               cudaStream_t s);
// Parts in which an adapter's second operand is checked (of about 64 KB), at
// most kCheckParts, the pitch of the maxima.
constexpr int kCheckParts = 32;
inline int check_parts(int64_t elements) {
  const int64_t n = (elements * 2 + 65535) / 65536;
  return n < kCheckParts ? static_cast<int>(n) : kCheckParts;
}
// Amax, row copy to nearest and decode scale of BF16 rows, without scale padding
// (operands.cu); `maxima`: kRowMaxima words of workspace.
constexpr int64_t kRowMaxima = 8 * 148;
cudaError_t launch_rows_operand(const void* x, int64_t ldx, int64_t T, int64_t K, void* maxima, void* data, void* scales,
                                float* gs, int num_sms, cudaStream_t s);
// After the shrink launch: the valid rows' row copy (sr:
// stochastic rounding) and its decode scale, without scale padding; and with
// `slabs` (E above) the slabs of the adapter tiles, V / alpha as two BF16 terms
// with alpha the product's decode scale.
cudaError_t launch_lora_operands(const void* x, int64_t ldx, int64_t T, int64_t K, int sr, uint64_t seed, void* data,
                                 void* scales, float* gs, const float* V, int64_t N, const LoraBatch& b, const LoraPlan& p,
                                 const float* gs_w, bool slabs, int num_sms, cudaStream_t s);
// A [count][rank][Cin] -> a_t [count][Cin][rank], B [count][Cout][rank] -> b_t
// [count][rank][Cout]; zeroes *amax; lists the rows of each adapter (sorted [T],
// span [count] = first in it, number).
cudaError_t launch_lora_transpose(const LoraBatch& b, const void* A, void* a_t, int64_t Cin, const void* B, void* b_t,
                                  int64_t Cout, int64_t T, float* amax, int* sorted, int2* span, cudaStream_t s);
// dA_i = sum over adapter i's rows of U[t, :]^T X[t, :] ([rank][Cin]) and dB_i =
// sum of dY[t, :]^T V[t, :] ([Cout][rank]), BF16; zeros where it has no rows.
cudaError_t launch_lora_grads(const float* U, const void* X, int64_t ldx, int64_t Cin, const float* V, const void* dY,
                              int64_t ldy, int64_t Cout, int64_t T, const LoraBatch& b, const int* sorted, const int2* span,
                              void* dA, void* dB, int num_sms, cudaStream_t s);

// Bounded-wait self-test: a kernel waits on an mbarrier nobody arrives on.
cudaError_t launch_wait_probe(uint32_t timeout_us, cudaStream_t s);

cudaError_t read_device_error(unsigned int* out, int clear);
cudaError_t read_project_error(unsigned int* out, int clear);   // project.cu's own word
cudaError_t read_rows_error(unsigned int* out, int clear);      // rows.cu's own word

}  // namespace nvfp4
