// api.cu -- the extern "C" boundary (include/nvfp4.h): argument checks, size
// queries, workspace layout and the linear-layer sequencing.  No kernel code
// here; every step of the path runs in the kernels of amax.cu, quantize.cu
// and gemm.cu.
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/nvfp4.h"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"

namespace {

using nvfp4::launch_amax;

inline int64_t pad128(int64_t v) { return (v + 127) / 128 * 128; }
inline int64_t pad4(int64_t v) { return (v + 3) / 4 * 4; }
inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct DeviceInfo {
  int sms = 0;
  bool ok = false;
};

// Per-device SM count and architecture check, queried once.
nvfp4_status device_info(DeviceInfo* out) {
  static std::mutex mu;
  static DeviceInfo cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return NVFP4_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev].ok) {
    int major = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    if (major != 10) return NVFP4_ERR_DEVICE;
    cache[dev].sms = sms;
    cache[dev].ok = true;
  }
  *out = cache[dev];
  return NVFP4_OK;
}

// Last CUDA error code behind an NVFP4_ERR_CUDA, per host thread.
thread_local int t_last_cuda_error = 0;

inline nvfp4_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return NVFP4_OK;
  t_last_cuda_error = static_cast<int>(e);
  return NVFP4_ERR_CUDA;
}

nvfp4_status check_tensor(const nvfp4_tensor* t, int64_t rows, int64_t cols) {
  if (!t || !t->data || !t->scales || !t->global_scale) return NVFP4_ERR_INVALID_ARG;
  if (t->rows != rows || t->cols != cols) return NVFP4_ERR_SHAPE;
  if (!aligned16(t->data) || !aligned16(t->scales) || (reinterpret_cast<uintptr_t>(t->global_scale) & 3))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// ---------------------------------------------------------------- workspace
constexpr int kWsTensors = 6;
struct WsLayout {
  int64_t rows[kWsTensors], cols[kWsTensors];
  size_t data[kWsTensors], scales[kWsTensors];
  size_t total;
};
// Scalars at offset 0: amax slots (floats 0..7), decode scales (floats 8..15).
// (kAmaxX, kAmaxXr) and (kAmaxDy, kAmaxDyr) are adjacent: one amax pass fills both.
enum { kAmaxX = 0, kAmaxXr = 1, kAmaxW = 2, kAmaxDy = 3, kAmaxDyr = 4 };

WsLayout ws_layout(int64_t T, int64_t Cin, int64_t Cout) {
  WsLayout L;
  const int64_t r[kWsTensors] = {T, Cout, Cin, Cin, T, Cout};
  const int64_t c[kWsTensors] = {Cin, Cin, Cout, T, Cout, T};
  size_t off = 256;
  for (int i = 0; i < kWsTensors; ++i) {
    L.rows[i] = r[i];
    L.cols[i] = c[i];
    L.data[i] = off;
    off = align256(off + static_cast<size_t>(r[i] * c[i] / 2));
    L.scales[i] = off;
    off = align256(off + static_cast<size_t>(pad128(r[i]) * pad4(c[i] / 16)));
  }
  L.total = off;
  return L;
}

nvfp4_tensor ws_tensor(void* ws, const WsLayout& L, int i) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  nvfp4_tensor t;
  t.data = b + L.data[i];
  t.scales = b + L.scales[i];
  t.global_scale = reinterpret_cast<float*>(b) + 8 + i;
  t.rows = L.rows[i];
  t.cols = L.cols[i];
  return t;
}

// Shape rules of the linear layer: multiples of 64, each below 2^31 (the GEMM
// limit), checked before any size arithmetic so ws_layout never overflows.
bool linear_shape_ok(int64_t T, int64_t Cin, int64_t Cout) {
  const int64_t lim = int64_t(1) << 31;
  return T > 0 && Cin > 0 && Cout > 0 && T < lim && Cin < lim && Cout < lim && T % 64 == 0 && Cin % 64 == 0 &&
         Cout % 64 == 0;
}

nvfp4_status linear_check(int64_t T, int64_t Cin, int64_t Cout, void* ws, size_t ws_bytes) {
  if (!linear_shape_ok(T, Cin, Cout)) return NVFP4_ERR_SHAPE;
  if (!ws || ws_bytes < ws_layout(T, Cin, Cout).total) return NVFP4_ERR_WORKSPACE;
  if (!aligned16(ws)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// A second stream of the library's own, one per device, created on first use
// (non-blocking), and two events per host thread and device, for the linear
// layer's independent branches.
nvfp4_status side_stream(int* dev_out, cudaStream_t* out) {
  static std::mutex mu;
  static cudaStream_t streams[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return NVFP4_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!streams[dev]) {
    cudaError_t e = cudaStreamCreateWithFlags(&streams[dev], cudaStreamNonBlocking);
    if (e != cudaSuccess) return cuda_status(e);
  }
  *dev_out = dev;
  *out = streams[dev];
  return NVFP4_OK;
}

// Fork: the side stream starts after the work enqueued on main so far.  Join:
// main continues after the work enqueued on the side stream since the fork.
// A stream wait binds to the event's latest record when it is enqueued, so a
// thread can re-record its two events in every call; calls from several host
// threads use different events.
struct Fork {
  cudaStream_t main = nullptr, side = nullptr;
  cudaEvent_t start = nullptr, done = nullptr;
};

nvfp4_status fork(cudaStream_t main, Fork* f) {
  thread_local cudaEvent_t events[64][2] = {};
  int dev = 0;
  nvfp4_status st = side_stream(&dev, &f->side);
  if (st != NVFP4_OK) return st;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2 && e == cudaSuccess; ++i)
    if (!events[dev][i]) e = cudaEventCreateWithFlags(&events[dev][i], cudaEventDisableTiming);
  if (e != cudaSuccess) return cuda_status(e);
  f->main = main;
  f->start = events[dev][0];
  f->done = events[dev][1];
  e = cudaEventRecord(f->start, main);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(f->side, f->start, 0);
  if (e != cudaSuccess) f->side = nullptr;      // nothing was forked
  return cuda_status(e);
}

nvfp4_status join(Fork* f) {
  if (!f->side) return NVFP4_OK;
  cudaError_t e = cudaEventRecord(f->done, f->side);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(f->main, f->done, 0);
  f->side = nullptr;
  return cuda_status(e);
}

// After an error on one branch: main still waits for what the side stream
// already holds, so the caller's buffers stay in use until both are done.
nvfp4_status fail(Fork* f, nvfp4_status st) {
  (void)join(f);
  return st;
}

}  // namespace

namespace nvfp4 {

size_t linear_forward_bytes(int64_t T, int64_t Cin, int64_t Cout) {
  if (!linear_shape_ok(T, Cin, Cout)) return 0;
  return ws_layout(T, Cin, Cout).data[3];   // tensors 0..2 and the scalars come first
}

// The quantized operands of a forward: X row and W copies, and with keep_wgrad
// the X column copy.
static nvfp4_status forward_operands(const void* X, const void* W, int64_t T, int64_t Cin, int64_t Cout, void* ws,
                                     bool keep_wgrad, nvfp4_stream_t stream) {
  const WsLayout L = ws_layout(T, Cin, Cout);
  float* amax = static_cast<float*>(ws);
  const nvfp4_tensor xr = ws_tensor(ws, L, 0), wr = ws_tensor(ws, L, 1), wc = ws_tensor(ws, L, 2);
  nvfp4_status st;
  // W's amax and 2D copies (RN) on the side stream while X's run on the caller's
  // stream (without the wgrad operand -- the allocation-free forward -- both run
  // on the caller's stream: it creates no stream or event)
  Fork f;
  cudaStream_t wstream = reinterpret_cast<cudaStream_t>(stream);
  if (keep_wgrad) {
    if ((st = fork(wstream, &f)) != NVFP4_OK) return st;
    wstream = f.side;
  }
  nvfp4_stream_t ws_ = reinterpret_cast<nvfp4_stream_t>(wstream);
  if ((st = nvfp4_amax(W, Cout, Cin, Cin, 0, amax + kAmaxW, ws_)) != NVFP4_OK ||
      (st = nvfp4_quantize(W, Cout, Cin, Cin, NVFP4_2D, 0, 0, 0, amax + kAmaxW, &wr, &wc, ws_)) != NVFP4_OK)
    return fail(&f, st);
  // one pass over X gives both its amax (row copy) and its RHT amax (column copy)
  if ((st = nvfp4_amax(X, T, Cin, Cin, 2, amax + kAmaxX, stream)) != NVFP4_OK) return fail(&f, st);
  if (keep_wgrad) {
    // the X row copy (fprop) and the X^T copy with the RHT along tokens, saved
    // for wgrad, from one read of X; amax + kAmaxX holds [max|X|, max|Q X|]
    const nvfp4_tensor xc = ws_tensor(ws, L, 3);
    if ((st = nvfp4_quantize(X, T, Cin, Cin, NVFP4_ROWCOL, 1, 0, 0, amax + kAmaxX, &xr, &xc, stream)) != NVFP4_OK)
      return fail(&f, st);
    return join(&f);
  }
  return nvfp4_quantize(X, T, Cin, Cin, NVFP4_ROW, 0, 0, 0, amax + kAmaxX, &xr, nullptr, stream);
}

nvfp4_status linear_forward(const void* X, const void* W, int64_t T, int64_t Cin, int64_t Cout, void* Y, void* ws,
                            bool keep_wgrad, nvfp4_stream_t stream) {
  const nvfp4_status st = forward_operands(X, W, T, Cin, Cout, ws, keep_wgrad, stream);
  if (st != NVFP4_OK) return st;
  const WsLayout L = ws_layout(T, Cin, Cout);
  const nvfp4_tensor xr = ws_tensor(ws, L, 0), wr = ws_tensor(ws, L, 1);
  return nvfp4_gemm(&xr, &wr, Y, NVFP4_OUT_BF16, Cout, stream);
}

}  // namespace nvfp4

extern "C" {

size_t nvfp4_data_bytes(int64_t rows, int64_t cols) {
  return (rows > 0 && cols > 0) ? static_cast<size_t>(rows * (cols / 2)) : 0;
}

size_t nvfp4_scale_bytes(int64_t rows, int64_t cols) {
  return (rows > 0 && cols > 0) ? static_cast<size_t>(pad128(rows) * pad4(cols / 16)) : 0;
}

size_t nvfp4_mx_scale_bytes(int64_t rows, int64_t cols) {
  return (rows > 0 && cols > 0) ? static_cast<size_t>(pad128(rows) * pad4(cols / 32)) : 0;
}

nvfp4_status nvfp4_mx_quantize(const void* x, int64_t R, int64_t C, int64_t ld, const nvfp4_tensor* out,
                               nvfp4_stream_t stream) {
  if (!x || !out) return NVFP4_ERR_INVALID_ARG;
  if (R <= 0 || C <= 0 || ld < C || C % 32) return NVFP4_ERR_SHAPE;
  if (!aligned16(x) || ld % 8) return NVFP4_ERR_ALIGN;
  nvfp4_status st;
  if ((st = check_tensor(out, R, C)) != NVFP4_OK) return st;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  return cuda_status(nvfp4::launch_mx_quant_row(x, R, C, ld, out->data, out->scales, out->global_scale, di.sms,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_mx_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, nvfp4_out_dtype out_dtype,
                           int64_t ldd, nvfp4_stream_t stream) {
  if (!A || !B || !D) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
  const int64_t M = A->rows, N = B->rows, K = A->cols;
  if (M <= 0 || N <= 0 || K <= 0 || B->cols != K) return NVFP4_ERR_SHAPE;
  if (K % 32 || N % 16 || ldd < N || M >= (1LL << 31) || N >= (1LL << 31) || K >= (1LL << 31))
    return NVFP4_ERR_SHAPE;
  nvfp4_status st;
  if ((st = check_tensor(A, M, K)) != NVFP4_OK || (st = check_tensor(B, N, K)) != NVFP4_OK) return st;
  if (!aligned16(D) || ldd % 8) return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  return cuda_status(nvfp4::launch_gemm(A->data, A->scales, A->global_scale, B->data, B->scales, B->global_scale,
                                        M, N, K, D, out_dtype == NVFP4_OUT_BF16, ldd, di.sms,
                                        reinterpret_cast<cudaStream_t>(stream), 1));
}

uint32_t nvfp4_rht_sign_mask(void) { return nvfp4::kRhtSignMask; }

nvfp4_status nvfp4_selftest_scale_division(uint64_t* bad_quotients, uint64_t* bad_codes) {
  if (!bad_quotients || !bad_codes) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo di;
  nvfp4_status st = device_info(&di);
  if (st != NVFP4_OK) return st;
  unsigned long long q = 0, c = 0;
  st = cuda_status(nvfp4::selftest_div6(&q, &c, di.sms));
  *bad_quotients = q;
  *bad_codes = c;
  return st;
}

nvfp4_status nvfp4_selftest_sr_rounding(uint64_t* mismatches, uint64_t* checked) {
  if (!mismatches || !checked) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo di;
  nvfp4_status st = device_info(&di);
  if (st != NVFP4_OK) return st;
  unsigned long long m = 0, c = 0;
  st = cuda_status(nvfp4::selftest_sr(&m, &c));
  *mismatches = m;
  *checked = c;
  return st;
}

int nvfp4_version(void) { return 1; }

int nvfp4_last_cuda_error(const char** name) {
  const int e = t_last_cuda_error;
  if (name) *name = cudaGetErrorName(static_cast<cudaError_t>(e));
  return e;
}

const char* nvfp4_status_string(nvfp4_status s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_ERR_SHAPE: return "shape breaks a divisibility rule";
    case NVFP4_ERR_ALIGN: return "pointer or pitch misaligned";
    case NVFP4_ERR_UNSUPPORTED: return "mode/flag combination not supported";
    case NVFP4_ERR_DEVICE: return "device is not sm_100";
    case NVFP4_ERR_CUDA: return "CUDA launch or driver call failed";
    case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
    case NVFP4_ERR_TIMEOUT: return "a kernel gave up on a bounded wait";
  }
  return "unknown status";
}

nvfp4_status nvfp4_amax(const void* x, int64_t R, int64_t C, int64_t ld, int rht, float* amax_dev,
                        nvfp4_stream_t stream) {
  if (!x || !amax_dev || rht < 0 || rht > 2) return NVFP4_ERR_INVALID_ARG;
  if (R < 0 || C < 0 || ld < C) return NVFP4_ERR_SHAPE;
  if (!aligned16(x) || (reinterpret_cast<uintptr_t>(amax_dev) & 3)) return NVFP4_ERR_ALIGN;
  if (rht && (R % 16 || C % 4)) return NVFP4_ERR_SHAPE;
  if (rht && ld % 4) return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  nvfp4_status st = device_info(&di);
  if (st != NVFP4_OK) return st;
  return cuda_status(launch_amax(x, R, C, ld, rht, amax_dev, di.sms,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

static nvfp4_status quantize_checked(const void* x, int64_t R, int64_t C, int64_t ld, nvfp4_mode mode, int rht,
                                     int sr, uint64_t seed, int64_t row0, const float* amax_dev,
                                     const nvfp4_tensor* row_out, const nvfp4_tensor* col_out,
                                     nvfp4_stream_t stream) {
  if (!x || !amax_dev) return NVFP4_ERR_INVALID_ARG;
  if (mode != NVFP4_ROW && mode != NVFP4_COL && mode != NVFP4_ROWCOL && mode != NVFP4_2D)
    return NVFP4_ERR_INVALID_ARG;
  if (R <= 0 || C <= 0 || ld < C) return NVFP4_ERR_SHAPE;
  if (!aligned16(x) || ld % 8) return NVFP4_ERR_ALIGN;
  if (rht && mode != NVFP4_COL && mode != NVFP4_ROWCOL) return NVFP4_ERR_UNSUPPORTED;
  if (sr && mode == NVFP4_2D) return NVFP4_ERR_UNSUPPORTED;
  if (row0 < 0 || row0 % 16 || row0 >= (int64_t(1) << 40)) return NVFP4_ERR_SHAPE;
  if (row0 && row0 + R > (int64_t(1) << 62) / C) return NVFP4_ERR_SHAPE;  // (row0 + R) * C stays in int64
  if (row0 && mode == NVFP4_2D) return NVFP4_ERR_UNSUPPORTED;
  const bool want_row = mode == NVFP4_ROW || mode == NVFP4_ROWCOL || (mode == NVFP4_2D && row_out);
  const bool want_col = mode == NVFP4_COL || mode == NVFP4_ROWCOL || (mode == NVFP4_2D && col_out);
  if (mode == NVFP4_2D && !want_row && !want_col) return NVFP4_ERR_INVALID_ARG;
  if (want_row && C % 16) return NVFP4_ERR_SHAPE;
  if (want_col && (R % 16 || C % 4)) return NVFP4_ERR_SHAPE;
  if (mode == NVFP4_2D && (R % 16 || C % 16)) return NVFP4_ERR_SHAPE;
  nvfp4_status st;
  if (want_row && (st = check_tensor(row_out, R, C)) != NVFP4_OK) return st;
  if (want_col && (st = check_tensor(col_out, C, R)) != NVFP4_OK) return st;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (mode == NVFP4_2D) {
    e = nvfp4::launch_quant_2d(x, R, C, ld, amax_dev, want_row ? row_out->data : nullptr,
                               want_row ? row_out->scales : nullptr, want_row ? row_out->global_scale : nullptr,
                               want_col ? col_out->data : nullptr, want_col ? col_out->scales : nullptr,
                               want_col ? col_out->global_scale : nullptr, di.sms, s);
    return cuda_status(e);
  }
  // ROWCOL with RHT: the row copy takes amax_dev[0], the RHT column copy amax_dev[1]
  const float* amax_col = (mode == NVFP4_ROWCOL && rht) ? amax_dev + 1 : amax_dev;
  if (mode == NVFP4_ROWCOL && !sr) {   // both copies from one read of x
    e = nvfp4::launch_quant_rowcol(x, R, C, ld, amax_dev, amax_col, rht, row_out->data, row_out->scales,
                                   row_out->global_scale, col_out->data, col_out->scales, col_out->global_scale,
                                   di.sms, s);
    return cuda_status(e);
  }
  if (want_row) {
    e = nvfp4::launch_quant_row(x, R, C, ld, amax_dev, sr, seed, row0 * C, row_out->data, row_out->scales,
                                row_out->global_scale, di.sms, s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (want_col) {
    e = nvfp4::launch_quant_col(x, R, C, ld, amax_col, rht, sr, seed, row0 * C, col_out->data,
                                col_out->scales, col_out->global_scale, di.sms, s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  return NVFP4_OK;
}

nvfp4_status nvfp4_quantize(const void* x, int64_t R, int64_t C, int64_t ld, nvfp4_mode mode, int rht, int sr,
                            uint64_t seed, const float* amax_dev, const nvfp4_tensor* row_out,
                            const nvfp4_tensor* col_out, nvfp4_stream_t stream) {
  return quantize_checked(x, R, C, ld, mode, rht, sr, seed, 0, amax_dev, row_out, col_out, stream);
}

nvfp4_status nvfp4_quantize_rows(const void* x, int64_t R, int64_t C, int64_t ld, nvfp4_mode mode, int rht,
                                 int sr, uint64_t seed, int64_t row0, const float* amax_dev,
                                 const nvfp4_tensor* row_out, const nvfp4_tensor* col_out, nvfp4_stream_t stream) {
  return quantize_checked(x, R, C, ld, mode, rht, sr, seed, row0, amax_dev, row_out, col_out, stream);
}

static nvfp4_status gemm_checked(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, nvfp4_out_dtype out_dtype,
                          int64_t ldd, float* amax_out, nvfp4_stream_t stream) {
  if (!A || !B || !D) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
  const int64_t M = A->rows, N = B->rows, K = A->cols;
  if (M <= 0 || N <= 0 || K <= 0 || B->cols != K) return NVFP4_ERR_SHAPE;
  if (K % 32 || N % 16 || ldd < N || M >= (1LL << 31) || N >= (1LL << 31) || K >= (1LL << 31))
    return NVFP4_ERR_SHAPE;
  nvfp4_status st;
  if ((st = check_tensor(A, M, K)) != NVFP4_OK || (st = check_tensor(B, N, K)) != NVFP4_OK) return st;
  if (!aligned16(D) || ldd % 8) return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  return cuda_status(nvfp4::launch_gemm(A->data, A->scales, A->global_scale, B->data, B->scales, B->global_scale,
                                        M, N, K, D, out_dtype == NVFP4_OUT_BF16, ldd, di.sms,
                                        reinterpret_cast<cudaStream_t>(stream), 0, amax_out));
}

nvfp4_status nvfp4_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, nvfp4_out_dtype out_dtype,
                        int64_t ldd, nvfp4_stream_t stream) {
  return gemm_checked(A, B, D, out_dtype, ldd, nullptr, stream);
}

nvfp4_status nvfp4_gemm_amax(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, nvfp4_out_dtype out_dtype,
                             int64_t ldd, float* amax_dev, nvfp4_stream_t stream) {
  if (!amax_dev) return NVFP4_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(amax_dev) % 4) return NVFP4_ERR_ALIGN;
  return gemm_checked(A, B, D, out_dtype, ldd, amax_dev, stream);
}

size_t nvfp4_linear_workspace_bytes(int64_t T, int64_t Cin, int64_t Cout) {
  const int64_t lim = int64_t(1) << 31;
  if (T <= 0 || Cin <= 0 || Cout <= 0 || T >= lim || Cin >= lim || Cout >= lim) return 0;
  return ws_layout(T, Cin, Cout).total;
}

nvfp4_status nvfp4_linear_workspace_tensor(void* workspace, int64_t T, int64_t Cin, int64_t Cout, int which,
                                           nvfp4_tensor* out) {
  if (!workspace || !out || which < 0 || which >= kWsTensors) return NVFP4_ERR_INVALID_ARG;
  const int64_t lim = int64_t(1) << 31;
  if (T <= 0 || Cin <= 0 || Cout <= 0 || T >= lim || Cin >= lim || Cout >= lim) return NVFP4_ERR_SHAPE;
  *out = ws_tensor(workspace, ws_layout(T, Cin, Cout), which);
  return NVFP4_OK;
}

nvfp4_status nvfp4_linear_fwd(const void* X, const void* W, int64_t T, int64_t Cin, int64_t Cout, void* Y,
                              void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!X || !W || !Y) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = linear_check(T, Cin, Cout, workspace, workspace_bytes);
  if (st != NVFP4_OK) return st;
  if (!aligned16(X) || !aligned16(W) || !aligned16(Y)) return NVFP4_ERR_ALIGN;
  return nvfp4::linear_forward(X, W, T, Cin, Cout, Y, workspace, true, stream);
}

nvfp4_status nvfp4_linear_bwd(const void* dY, int64_t T, int64_t Cin, int64_t Cout, uint64_t seed, void* dX,
                              float* dW, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!dY || !dX || !dW) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = linear_check(T, Cin, Cout, workspace, workspace_bytes);
  if (st != NVFP4_OK) return st;
  if (!aligned16(dY) || !aligned16(dX) || !aligned16(dW)) return NVFP4_ERR_ALIGN;
  const WsLayout L = ws_layout(T, Cin, Cout);
  float* amax = static_cast<float*>(workspace);
  const nvfp4_tensor wc = ws_tensor(workspace, L, 2), xc = ws_tensor(workspace, L, 3),
                     gr = ws_tensor(workspace, L, 4), gc = ws_tensor(workspace, L, 5);
  // one pass over dY gives both its amax (row copy) and its RHT amax (column copy)
  if ((st = nvfp4_amax(dY, T, Cout, Cout, 2, amax + kAmaxDy, stream)) != NVFP4_OK) return st;
  // wgrad: dW = dY^T X, both with the RHT along tokens, SR on dY
  if ((st = nvfp4_quantize(dY, T, Cout, Cout, NVFP4_COL, 1, 1, seed, amax + kAmaxDyr, nullptr, &gc, stream)) !=
      NVFP4_OK)
    return st;
  // the dY row copy (SR) for dgrad on the side stream, next to the wgrad GEMM:
  // the quantizer is bound by the integer ALU pipe, the GEMM by the tensor pipe,
  // and its CTAs fit beside the GEMM's on every SM
  Fork f;
  if ((st = fork(reinterpret_cast<cudaStream_t>(stream), &f)) != NVFP4_OK) return st;
  if ((st = nvfp4_gemm(&gc, &xc, dW, NVFP4_OUT_F32, Cin, stream)) != NVFP4_OK ||
      (st = nvfp4_quantize(dY, T, Cout, Cout, NVFP4_ROW, 0, 1, seed, amax + kAmaxDy, &gr, nullptr,
                           reinterpret_cast<nvfp4_stream_t>(f.side))) != NVFP4_OK)
    return fail(&f, st);
  if ((st = join(&f)) != NVFP4_OK) return st;
  // dgrad: dX = dY W, dY row-wise with SR, W^T from the 2D column copy
  return nvfp4_gemm(&gr, &wc, dX, NVFP4_OUT_BF16, Cin, stream);
}

// ---------------------------------------------------------------- gated projection
static bool act_ok(nvfp4_activation act) { return act == NVFP4_ACT_SILU || act == NVFP4_ACT_GELU_TANH; }

static nvfp4::FpOperand operand(const nvfp4_tensor& t) {
  return nvfp4::FpOperand{static_cast<const uint8_t*>(t.data), static_cast<const uint8_t*>(t.scales), t.global_scale};
}

nvfp4_status nvfp4_gated_gemm(const nvfp4_tensor* A, const nvfp4_tensor* W, nvfp4_activation act, void* H, int64_t ldh,
                              void* GU, float* amax_dev, nvfp4_stream_t stream) {
  if (!A || !W || !H || !act_ok(act)) return NVFP4_ERR_INVALID_ARG;
  const int64_t M = A->rows, F = W->rows / 2, K = A->cols, lim = int64_t(1) << 31;
  if (M <= 0 || W->rows <= 0 || K <= 0 || W->cols != K || W->rows % 256 || K % 64 || ldh < F || M >= lim ||
      W->rows >= lim || K >= lim)
    return NVFP4_ERR_SHAPE;
  nvfp4_status st;
  if ((st = check_tensor(A, M, K)) != NVFP4_OK || (st = check_tensor(W, W->rows, K)) != NVFP4_OK) return st;
  if (!aligned16(H) || ldh % 8 || (GU && !aligned16(GU)) || (reinterpret_cast<uintptr_t>(amax_dev) & 3))
    return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  return cuda_status(nvfp4::launch_gated_tiles(operand(*A), operand(*W), M, F, K, act, H, ldh, GU, amax_dev, di.sms,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

// Workspace of nvfp4_gated_apply: decode scale, maxima, then X's row copy.
// C below 2^24: the quantizer of few rows counts their blocks in 32 bits.
constexpr int64_t kApplyColumns = int64_t(1) << 24;
static size_t apply_header() { return 256 + align256(nvfp4::kRowMaxima * 4); }
size_t nvfp4_gated_apply_workspace_bytes(int64_t T, int64_t C) {
  const int64_t lim = int64_t(1) << 31;
  if (T <= 0 || C <= 0 || T >= lim || C >= kApplyColumns) return 0;
  return apply_header() + align256(nvfp4_data_bytes(T, C)) + align256(nvfp4_scale_bytes(T, C));
}

nvfp4_status nvfp4_gated_apply(const void* X, int64_t T, int64_t ldx, const nvfp4_tensor* W, nvfp4_activation act, void* H,
                               int64_t ldh, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!W || !act_ok(act)) return NVFP4_ERR_INVALID_ARG;
  const int64_t C = W->cols, F = W->rows / 2, lim = int64_t(1) << 31;
  if (T < 0 || T >= lim || C <= 0 || C >= kApplyColumns || C % 64 || W->rows <= 0 || W->rows >= lim || W->rows % 256 || ldx < C ||
      ldh < F)
    return NVFP4_ERR_SHAPE;
  nvfp4_status st;
  if ((st = check_tensor(W, W->rows, C)) != NVFP4_OK) return st;
  if (T == 0) return NVFP4_OK;
  if (!X || !H) return NVFP4_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < nvfp4_gated_apply_workspace_bytes(T, C)) return NVFP4_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(H) || !aligned16(workspace) || ldx % 8 || ldh % 8) return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* data = ws + apply_header();
  const nvfp4_tensor xq{data, data + align256(nvfp4_data_bytes(T, C)), static_cast<float*>(workspace), T, C};
  if (T <= nvfp4::kFewRows) {
    st = cuda_status(nvfp4::launch_quant_few_rows(X, T, C, ldx, xq.data, xq.scales, xq.global_scale, s));
    if (st != NVFP4_OK) return st;
    return cuda_status(nvfp4::launch_gated_rows(operand(xq), operand(*W), T, F, C, act, H, ldh, di.sms, s));
  }
  st = cuda_status(
      nvfp4::launch_rows_operand(X, ldx, T, C, ws + 256, xq.data, xq.scales, xq.global_scale, di.sms, s));
  if (st != NVFP4_OK) return st;
  return nvfp4_gated_gemm(&xq, W, act, H, ldh, nullptr, nullptr, stream);
}

// The operands of a gated projection are those of a linear layer with Cout = 2F.
// F below 2^24: offsets in a 64-row tile stay in 32 bits.  Fewer than 2^36
// gradients: their blocks are counted in 32 bits (more of them, with dH, do not
// fit in 180 GB).
static bool gated_sizes_ok(int64_t T, int64_t F) {
  return F > 0 && F < (int64_t(1) << 24) && T < (int64_t(1) << 31) && T * 2 * F < (int64_t(1) << 36);
}
static nvfp4_status gated_check(int64_t T, int64_t C, int64_t F, nvfp4_activation act, void* ws, size_t ws_bytes) {
  if (!act_ok(act)) return NVFP4_ERR_INVALID_ARG;
  if (!gated_sizes_ok(T, F) || F % 128) return NVFP4_ERR_SHAPE;
  return linear_check(T, C, 2 * F, ws, ws_bytes);
}

size_t nvfp4_gated_workspace_bytes(int64_t T, int64_t C, int64_t F) {
  return gated_sizes_ok(T, F) ? nvfp4_linear_workspace_bytes(T, C, 2 * F) : 0;
}

nvfp4_status nvfp4_gated_fwd(const void* X, const void* W, int64_t T, int64_t C, int64_t F, nvfp4_activation act, void* H,
                             void* GU, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!X || !W || !H || !GU) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = gated_check(T, C, F, act, workspace, workspace_bytes);
  if (st != NVFP4_OK) return st;
  if (!aligned16(X) || !aligned16(W) || !aligned16(H) || !aligned16(GU)) return NVFP4_ERR_ALIGN;
  if ((st = nvfp4::forward_operands(X, W, T, C, 2 * F, workspace, true, stream)) != NVFP4_OK) return st;
  const WsLayout L = ws_layout(T, C, 2 * F);
  const nvfp4_tensor xr = ws_tensor(workspace, L, 0), wr = ws_tensor(workspace, L, 1);
  return nvfp4_gated_gemm(&xr, &wr, act, H, F, GU, nullptr, stream);
}

nvfp4_status nvfp4_gated_bwd(const void* dH, const void* GU, int64_t T, int64_t C, int64_t F, nvfp4_activation act,
                             uint64_t seed, void* dX, void* dW, nvfp4_out_dtype dw_dtype, void* workspace,
                             size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!dH || !GU || !dX || !dW) return NVFP4_ERR_INVALID_ARG;
  if (dw_dtype != NVFP4_OUT_F32 && dw_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = gated_check(T, C, F, act, workspace, workspace_bytes);
  if (st != NVFP4_OK) return st;
  if (!aligned16(dH) || !aligned16(GU) || !aligned16(dX) || !aligned16(dW)) return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  const WsLayout L = ws_layout(T, C, 2 * F);
  float* amax = static_cast<float*>(workspace);
  const nvfp4_tensor wc = ws_tensor(workspace, L, 2), xc = ws_tensor(workspace, L, 3), gr = ws_tensor(workspace, L, 4),
                     gc = ws_tensor(workspace, L, 5);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((st = cuda_status(nvfp4::launch_gated_grad_amax(dH, GU, T, F, act, amax + kAmaxDy, di.sms, s))) != NVFP4_OK ||
      (st = cuda_status(nvfp4::launch_gated_grad_quant(dH, GU, T, F, act, amax + kAmaxDy, seed, gr.data, gr.scales,
                                                       gr.global_scale, gc.data, gc.scales, gc.global_scale, di.sms, s))) !=
          NVFP4_OK)
    return st;
  // Both products at once: one fills the SMs that the other's last wave leaves
  // (1088 x 1088 by 2 x 8832 107 us one after the other, 93 so; 8192 x 5120 by
  // 2 x 10240 the same).
  Fork f;
  if ((st = fork(s, &f)) != NVFP4_OK) return st;
  if ((st = nvfp4_gemm(&gr, &wc, dX, NVFP4_OUT_BF16, C, reinterpret_cast<nvfp4_stream_t>(f.side))) != NVFP4_OK ||
      (st = nvfp4_gemm(&gc, &xc, dW, dw_dtype, C, stream)) != NVFP4_OK)
    return fail(&f, st);
  return join(&f);
}

// ---------------------------------------------------------------- low-rank adapters
// Workspace of the adapter calls: scalars, plan, V or U, slabs, the operand's
// row copy and, for the backward, the transposed adapters and the lists of rows.
struct LoraLayout {
  size_t tile_count, tile_base, slab_adapter, slab_source, row_adapter, tile_direct, second_max, v, slabs, data, scales, a_t, b_t, sorted, span, total;
};
// Few rows and ranks: the kernel that streams W and adds the low-rank products
// row by row, 16 ranks at a time, each CTA of a tile those of its share of the
// rows.  Measured against tiles of 256 rows, 24 adapters, us by rows and by
// tiles: 4096 x 4096 (8 CTAs a tile) rank 16, 128 rows 21 and 33; rank 64, 64
// rows 31 and 37, 128 rows 53 and 44; 256 x 4096 (one CTA) rank 16, 32 rows 12
// and 23, 128 rows 36 and 25; 8192 x 8192 (4 CTAs) rank 16, 128 rows 28 and 43,
// rank 128, 32 rows 60 and 92, 64 rows 99 and 86.
// (The layout is made without a device: the 148 SMs of a B200.)
static bool lora_few(int64_t T, int64_t rank, int64_t N, int64_t K) {
  if (T > nvfp4::kFewRows) return false;
  const int64_t slices = nvfp4::rows_slices((N + 127) / 128, (K + 255) / 256, 148);
  return (T + slices - 1) / slices * (rank < 16 ? 16 : rank) / 8 <= (N * K < (int64_t(1) << 25) ? 96 : 128);
}

// K: the columns of the quantized operand (X in the forward, dY in the backward).
static LoraLayout lora_layout(int64_t T, int64_t S, int64_t count, int64_t rank, int64_t K, int64_t N, bool backward) {
  LoraLayout L;
  size_t off = 256;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off = align256(off + static_cast<size_t>(bytes));
    return at;
  };
  const int64_t tiles = (T + 255) / 256, slabs = lora_few(T, rank, N, K) ? 0 : S + tiles;
  L.tile_count = take(tiles * 4);
  L.tile_base = take(tiles * 4);
  L.slab_adapter = take(slabs * 4);
  L.slab_source = take(slabs * 4);
  L.row_adapter = take(T * 4);
  L.tile_direct = take(tiles * 4);
  L.second_max = take(slabs ? count * 32 * 4 : 0);
  L.v = take(T * rank * 4);
  L.slabs = take(slabs * 256 * ((rank + 31) / 32 * 32) * 2 * 2);   // two BF16 terms
  L.data = take(T * (K / 2));
  L.scales = take(pad128(T) * pad4(K / 16));
  L.a_t = take(backward ? count * rank * N * 2 : 0);
  L.b_t = take(backward ? count * rank * K * 2 : 0);
  L.sorted = take(backward ? T * 4 : 0);
  L.span = take(backward ? count * 8 : 0);
  L.total = off;
  return L;
}

// Sizes below these bounds keep every index of the kernels in its type and the
// layout's bytes in 64 bits.
static bool lora_sizes_ok(int64_t T, int64_t S, int64_t count, int64_t rank, int64_t Cin, int64_t Cout) {
  const int64_t lim = int64_t(1) << 31;
  return T >= 0 && T < (int64_t(1) << 30) && S >= 0 && S < (int64_t(1) << 24) && count > 0 && count < 65536 && rank >= 8 &&
         rank <= 128 && rank % 8 == 0 && Cin > 0 && Cout > 0 && Cin < (int64_t(1) << 20) && Cout < (int64_t(1) << 20) &&
         Cin % 64 == 0 && Cout % 64 == 0 && (count + 1) * Cin < lim && (count + 1) * Cout < lim && (S + T / 256 + 1) * 256 < lim;
}

static size_t lora_bytes(int64_t T, int64_t S, int64_t count, int64_t rank, int64_t Cin, int64_t Cout, bool backward) {
  if (T <= 0 || !lora_sizes_ok(T, S, count, rank, Cin, Cout)) return 0;
  return backward ? lora_layout(T, S, count, rank, Cout, Cin, true).total
                  : lora_layout(T, S, count, rank, Cin, Cout, false).total;
}

size_t nvfp4_lora_workspace_bytes(int64_t T, int64_t S, int64_t count, int64_t rank, int64_t Cin, int64_t Cout,
                                  int backward) {
  return lora_bytes(T, S, count, rank, Cin, Cout, backward != 0);
}

static nvfp4_status adapters_check(const nvfp4_adapters* ad, const int32_t* seg_ptr, const int32_t* seg_adapter, int64_t S) {
  if (!ad || !ad->A || !ad->B || !ad->scale || (S > 0 && (!seg_ptr || !seg_adapter))) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(ad->A) || !aligned16(ad->B) ||
      ((reinterpret_cast<uintptr_t>(ad->scale) | reinterpret_cast<uintptr_t>(seg_ptr) |
        reinterpret_cast<uintptr_t>(seg_adapter)) & 3))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Where the adapters' gradients go (backward only), and what they are made of
// besides v and x.
struct LoraGrads {
  const void* X;
  int64_t ldx;
  const float* V;
  const int* sorted;   // the rows of each adapter
  const int2* span;
  void* dA;
  void* dB;
};

// out[t] = x[t] W^T + v[t] (expand_i)^T, v = scale_i x[t] (shrink_i)^T: the
// forward with (A, B), the backward's dX with the transposed (B, A) and
// stochastic rounding of x = dY.  With `grads` (backward) also dA and dB, which
// need nothing but v, x, X and V.
static nvfp4_status lora_project(const void* x, int64_t T, int64_t ldx, const nvfp4_tensor& W, const void* shrink,
                                 const void* expand, const nvfp4::LoraBatch& b, const LoraGrads* grads, uint64_t seed,
                                 float* v, uint8_t* ws, const LoraLayout& L, void* out, int64_t ldo, int sms,
                                 cudaStream_t s) {
  using namespace nvfp4;
  const int64_t N = W.rows, K = W.cols;
  float* scalars = reinterpret_cast<float*>(ws);
  LoraPlan plan;
  plan.valid_rows = reinterpret_cast<int*>(ws) + 2;
  plan.tile_count = reinterpret_cast<int*>(ws + L.tile_count);
  plan.tile_base = reinterpret_cast<int*>(ws + L.tile_base);
  plan.slab_adapter = reinterpret_cast<int*>(ws + L.slab_adapter);
  plan.slab_source = reinterpret_cast<int*>(ws + L.slab_source);
  plan.row_adapter = reinterpret_cast<int*>(ws + L.row_adapter);
  plan.tile_direct = reinterpret_cast<int*>(ws + L.tile_direct);
  plan.second_max = reinterpret_cast<int*>(ws + L.second_max);
  plan.slabs = ws + L.slabs;
  plan.amax = scalars;
  const FpOperand xq{ws + L.data, ws + L.scales, scalars + 1};
  float* gs = scalars + 1;
  const int sr = grads != nullptr;
  auto gradients = [&](cudaStream_t on) {
    return grads ? launch_lora_grads(v, grads->X, grads->ldx, N, grads->V, x, ldx, K, T, b, grads->sorted, grads->span, grads->dA,
                                     grads->dB, sms, on)
                 : cudaSuccess;
  };
  cudaError_t e;
  if (lora_few(T, b.rank, N, K)) {
    // a block for each row and eight ranks beside the quantizer, then the kernel for few rows
    e = launch_lora_few_rows(x, T, K, ldx, sr, seed, ws + L.data, ws + L.scales, gs, shrink, b, plan.row_adapter, v, s);
    if (e == cudaSuccess)
      e = launch_adapter_rows(xq, operand(W), T, N, K, plan.row_adapter, v, expand, b.rank, out, ldo, sms, s);
    if (e == cudaSuccess) e = gradients(s);
    return cuda_status(e);
  }
  // Tiles of 256 rows cost a K step for each adapter in the tile.  With very many
  // adapters in a middling batch 128 rows at a time take less, by the kernel for
  // few rows, which adds each row's low-rank product by itself.
  const int64_t adapters = b.S < b.count ? b.S : b.count;
  const bool by_rows = T <= 2 * kFewRows && T * (b.rank / 8) <= 1024 && adapters > 96;
  // the backward's transposing launch has zeroed the amax
  if ((e = launch_lora_shrink(x, ldx, T, K, shrink, by_rows ? nullptr : expand, N, b, plan, grads != nullptr, v, sms, s)) !=
      cudaSuccess)
    return cuda_status(e);
  // dA and dB read memory while dX's product uses the tensor cores: beside it
  // on the side stream, where the work is worth two events (2^28 products with
  // V and U, about 10 us)
  const bool beside = grads && static_cast<double>(T) * (N + K) * b.rank >= 268435456.0;
  Fork f;
  nvfp4_status st;
  if (beside) {
    if ((st = fork(s, &f)) != NVFP4_OK) return st;
    if ((e = gradients(f.side)) != cudaSuccess) return fail(&f, cuda_status(e));
  }
  e = launch_lora_operands(x, ldx, T, K, sr, seed, ws + L.data, ws + L.scales, gs, v, N, b, plan, W.global_scale, !by_rows, sms,
                           s);
  if (e != cudaSuccess) return fail(&f, cuda_status(e));
  for (int64_t t = 0; by_rows && t < T; t += kFewRows) {
    const FpOperand part{xq.data + t * (K / 2), xq.scales + t * (K / 16), gs};   // 128 rows are whole scale tiles
    e = launch_adapter_rows(part, operand(W), T - t < kFewRows ? T - t : kFewRows, N, K, plan.row_adapter + t,
                            v + t * b.rank, expand, b.rank, static_cast<uint8_t*>(out) + t * ldo * 2, ldo, sms, s);
    if (e != cudaSuccess) return fail(&f, cuda_status(e));
  }
  if (by_rows) return beside ? join(&f) : cuda_status(gradients(s));
  AdapterPlan ap{plan.valid_rows, plan.tile_count, plan.tile_base, plan.slab_source, plan.slabs,
                 b.S + (T + 255) / 256, plan.tile_direct, v, plan.row_adapter};
  e = launch_adapter_tiles(xq, operand(W), T, N, K, ap, expand, b.count, b.rank, out, ldo, sms, s);
  if (e != cudaSuccess) return fail(&f, cuda_status(e));
  if (beside) return join(&f);
  return cuda_status(gradients(s));
}

nvfp4_status nvfp4_lora_fwd(const void* X, int64_t T, int64_t ldx, const nvfp4_tensor* W, const nvfp4_adapters* ad,
                            const int32_t* seg_ptr, const int32_t* seg_adapter, int64_t S, void* Y, int64_t ldy, float* V,
                            void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!W) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = adapters_check(ad, seg_ptr, seg_adapter, S);
  if (st != NVFP4_OK) return st;
  const int64_t N = W->rows, K = W->cols;
  if (!lora_sizes_ok(T, S, ad->count, ad->rank, K, N) || ldx < K || ldy < N) return NVFP4_ERR_SHAPE;
  if ((st = check_tensor(W, N, K)) != NVFP4_OK) return st;
  if (T == 0 || S == 0) return NVFP4_OK;
  if (!X || !Y) return NVFP4_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < lora_bytes(T, S, ad->count, ad->rank, K, N, false)) return NVFP4_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(workspace) || ldx % 8 || ldy % 8 || (V && !aligned16(V)))
    return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  const LoraLayout L = lora_layout(T, S, ad->count, ad->rank, K, N, false);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const nvfp4::LoraBatch b{seg_ptr, seg_adapter, static_cast<int>(S), ad->scale, static_cast<int>(ad->count),
                           static_cast<int>(ad->rank)};
  return lora_project(X, T, ldx, *W, ad->A, ad->B, b, nullptr, 0, V ? V : reinterpret_cast<float*>(ws + L.v), ws, L, Y, ldy,
                      di.sms, reinterpret_cast<cudaStream_t>(stream));
}

nvfp4_status nvfp4_lora_bwd(const void* dY, int64_t ldy, const void* X, int64_t ldx, const float* V, int64_t T,
                            const nvfp4_tensor* W, const nvfp4_adapters* ad, const int32_t* seg_ptr,
                            const int32_t* seg_adapter, int64_t S, uint64_t seed, void* dX, int64_t lddx, void* dA, void* dB,
                            void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!W || !dA || !dB) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = adapters_check(ad, seg_ptr, seg_adapter, S);
  if (st != NVFP4_OK) return st;
  const int64_t Cin = W->rows, Cout = W->cols;
  if (!lora_sizes_ok(T, S, ad->count, ad->rank, Cin, Cout) || ldx < Cin || lddx < Cin || ldy < Cout) return NVFP4_ERR_SHAPE;
  if ((st = check_tensor(W, Cin, Cout)) != NVFP4_OK) return st;
  if (!aligned16(dA) || !aligned16(dB)) return NVFP4_ERR_ALIGN;
  DeviceInfo di;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0 || S == 0) {   // no rows: zero gradients of the adapters
    const size_t row = static_cast<size_t>(ad->count * ad->rank) * 2;
    if ((st = device_info(&di)) != NVFP4_OK) return st;
    cudaError_t e = cudaMemsetAsync(dA, 0, row * static_cast<size_t>(Cin), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, row * static_cast<size_t>(Cout), s);
    return cuda_status(e);
  }
  if (!dY || !X || !V || !dX) return NVFP4_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < lora_bytes(T, S, ad->count, ad->rank, Cin, Cout, true)) return NVFP4_ERR_WORKSPACE;
  if (!aligned16(dY) || !aligned16(X) || !aligned16(V) || !aligned16(dX) || !aligned16(workspace) || ldy % 8 || ldx % 8 ||
      lddx % 8)
    return NVFP4_ERR_ALIGN;
  if ((st = device_info(&di)) != NVFP4_OK) return st;
  const LoraLayout L = lora_layout(T, S, ad->count, ad->rank, Cout, Cin, true);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const nvfp4::LoraBatch b{seg_ptr, seg_adapter, static_cast<int>(S), ad->scale, static_cast<int>(ad->count),
                           static_cast<int>(ad->rank)};
  // both products of the projection contract the innermost index: B^T [r, Cout] and A^T [Cin, r]
  const cudaError_t e =
      nvfp4::launch_lora_transpose(b, ad->A, ws + L.a_t, Cin, ad->B, ws + L.b_t, Cout, T, reinterpret_cast<float*>(ws),
                                   reinterpret_cast<int*>(ws + L.sorted), reinterpret_cast<int2*>(ws + L.span), s);
  if (e != cudaSuccess) return cuda_status(e);
  const LoraGrads grads{X,  ldx, V, reinterpret_cast<const int*>(ws + L.sorted), reinterpret_cast<const int2*>(ws + L.span),
                        dA, dB};
  return lora_project(dY, T, ldy, *W, ws + L.b_t, ws + L.a_t, b, &grads, seed, reinterpret_cast<float*>(ws + L.v), ws, L, dX,
                      lddx, di.sms, s);
}

// The library's error word and those of the units that keep their own: the
// first one that is set.
nvfp4_status nvfp4_read_device_error(unsigned int* code, int clear) {
  if (!code) return NVFP4_ERR_INVALID_ARG;
  unsigned int words[3] = {0, 0, 0};
  cudaError_t e = nvfp4::read_device_error(&words[0], clear);
  if (e == cudaSuccess) e = nvfp4::read_project_error(&words[1], clear);
  if (e == cudaSuccess) e = nvfp4::read_rows_error(&words[2], clear);
  if (e == cudaSuccess) *code = words[0] ? words[0] : words[1] ? words[1] : words[2];
  return cuda_status(e);
}

nvfp4_status nvfp4_wait_probe(uint32_t timeout_us, nvfp4_stream_t stream) {
  DeviceInfo di;
  nvfp4_status st = device_info(&di);
  if (st != NVFP4_OK) return st;
  return cuda_status(nvfp4::launch_wait_probe(timeout_us, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
