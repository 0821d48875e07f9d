// C ABI of libfp4lin.so: argument checks, workspace layout and launches.
// Every check runs on the host before anything is enqueued; no call allocates,
// frees, synchronises or reads device memory.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fp4lin.h"
#include "internal.hpp"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;

bool bad_dtype(fp4lin_dtype dt) { return dt != FP4LIN_F32 && dt != FP4LIN_BF16; }
// histogram bins count in 32 bits
constexpr int64_t kMaxCount = int64_t(1) << 32;
bool ok_dim(int64_t x) { return x >= 1 && x < kMaxDim; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// HIP error behind the calling thread's last launch check (for
// fp4lin_last_hip_error).
thread_local hipError_t t_last_hip = hipSuccess;

fp4lin_status launch_status(hipError_t e) {
  t_last_hip = e;
  return e == hipSuccess ? FP4LIN_OK : FP4LIN_ERR_LAUNCH;
}

// The micro-scaled column quantizer launches one workgroup row per 128 codes
// of K along the grid's second dimension, which holds at most 65535; the
// token-wise one keeps the same limit.
constexpr int64_t kMaxColK = int64_t(65535) * 128;

// The column quantizers' one-dimensional grids (128-column tiles by 64 rows at
// the finest, plus the select's row workgroups when they share a launch) fit
// the 32-bit workgroup count.
bool col_grids_fit(int64_t K, int64_t N) {
  return ((N + 127) / 128) * ((K + 63) / 64) < (int64_t(1) << 32) - 4096;
}

// COO entries the select can produce for rank k: #{|a| > tau} <= n - 1 - k.
int64_t needed_capacity(int64_t n, int64_t k) { return n - 1 - k; }

size_t weight_ws(int64_t N) { return round_up(fp4lin::weight_workspace_bytes(N), 256); }

// The compensation kernel addresses W with 32-bit byte offsets.
bool weight_addressable(int64_t K, int64_t ldw, fp4lin_dtype wdt) {
  return K * ldw * (wdt == FP4LIN_BF16 ? 2 : 4) < kMaxDim;
}

size_t select_ws(int64_t M, fp4lin_dtype dt) {
  return round_up(fp4lin::select_workspace_bytes(dt == FP4LIN_BF16, M), 256);
}

}  // namespace

extern "C" {

int64_t fp4lin_quantile_rank(int64_t n, double q) {
  if (n < 1 || !(q >= 0.0 && q <= 1.0)) return -1;
  const double c = std::ceil(q * double(n));
  int64_t k = int64_t(c) - 1;
  if (k < 0) k = 0;
  if (k > n - 1) k = n - 1;
  return k;
}

int64_t fp4lin_packed_ld(int64_t L) {
  if (L < 1) return -1;
  return (L + 127) / 128 * 64;
}

size_t fp4lin_select_workspace_bytes(int64_t M, int64_t K, fp4lin_dtype dt) {
  if (!ok_dim(M) || !ok_dim(K) || bad_dtype(dt)) return 0;
  return select_ws(M, dt);
}

size_t fp4lin_weight_workspace_bytes(int64_t K, int64_t N) {
  if (!ok_dim(K) || !ok_dim(N)) return 0;
  return weight_ws(N);
}

}  // extern "C"

namespace {

// The forward's workspace: tau, the COO, the packed operands with their
// scales (fp32 vectors, or with mx the step-major E8M0 block scales), then
// scratch.
fp4lin_status forward_layout(int64_t M, int64_t K, int64_t N, fp4lin_dtype dt, double q, bool mx,
                             fp4lin_forward_offsets* out) {
  if (out == nullptr) return FP4LIN_ERR_NULL;
  if (!ok_dim(M) || !ok_dim(K) || !ok_dim(N)) return FP4LIN_ERR_SHAPE;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  const int64_t n = M * K;
  if (n >= kMaxCount) return FP4LIN_ERR_SHAPE;
  const int64_t k = fp4lin_quantile_rank(n, q);
  if (k < 0) return FP4LIN_ERR_QUANTILE;
  const int64_t cap = needed_capacity(n, k);
  if (cap >= kMaxDim) return FP4LIN_ERR_SHAPE;
  const size_t slots = size_t(cap > 0 ? cap : 1);
  const size_t ldq = size_t(fp4lin_packed_ld(K));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  fp4lin_forward_offsets o{};
  o.tau = take(4);
  o.coo_row = take(slots * 4);
  o.coo_col = take(slots * 4);
  o.coo_val = take(slots * 4);
  o.row_ptr = take(size_t(M + 1) * 4);
  const size_t nblk = ldq / 16;
  o.Aq = take(size_t(M) * ldq);
  o.sA = take(size_t(M) * (mx ? nblk : 4));
  o.Wq = take(size_t(N) * ldq);
  o.sW = take(size_t(N) * (mx ? nblk : 4));
  // the select's workspace, then (token-wise) the column maxima of W's
  // quantization: the forward keeps both live at once
  o.scratch = take(select_ws(M, dt) + (mx ? 0 : weight_ws(N)));
  o.capacity = cap;
  o.total = off;
  *out = o;
  return FP4LIN_OK;
}

}  // namespace

extern "C" {

fp4lin_status fp4lin_forward_layout(int64_t M, int64_t K, int64_t N, fp4lin_dtype dt, double q,
                                    fp4lin_forward_offsets* out) {
  return forward_layout(M, K, N, dt, q, false, out);
}

fp4lin_status fp4lin_forward_layout_mx(int64_t M, int64_t K, int64_t N, fp4lin_dtype dt,
                                       double q, fp4lin_forward_offsets* out) {
  return forward_layout(M, K, N, dt, q, true, out);
}

size_t fp4lin_workspace_bytes(int64_t M, int64_t K, int64_t N, fp4lin_dtype dt, double q) {
  fp4lin_forward_offsets o;
  if (fp4lin_forward_layout(M, K, N, dt, q, &o) != FP4LIN_OK) return 0;
  return o.total;
}

size_t fp4lin_workspace_bytes_mx(int64_t M, int64_t K, int64_t N, fp4lin_dtype dt, double q) {
  fp4lin_forward_offsets o;
  if (fp4lin_forward_layout_mx(M, K, N, dt, q, &o) != FP4LIN_OK) return 0;
  return o.total;
}

int fp4lin_last_hip_error(void) { return int(t_last_hip); }

const char* fp4lin_last_hip_error_name(void) { return hipGetErrorName(t_last_hip); }

const char* fp4lin_status_str(fp4lin_status s) {
  switch (s) {
    case FP4LIN_OK: return "ok";
    case FP4LIN_ERR_NULL: return "a required pointer is NULL";
    case FP4LIN_ERR_SHAPE: return "invalid shape or leading dimension";
    case FP4LIN_ERR_DTYPE: return "unsupported dtype";
    case FP4LIN_ERR_QUANTILE: return "quantile q must be in [0, 1]";
    case FP4LIN_ERR_CAPACITY: return "COO capacity below M*K - 1 - k";
    case FP4LIN_ERR_ALIGN: return "pointer not 16-byte aligned";
    case FP4LIN_ERR_WORKSPACE: return "workspace too small";
    case FP4LIN_ERR_LAUNCH: return "kernel launch failed";
    case FP4LIN_ERR_SCRATCH: return "input needs more than the static scratch of the allocation-free call";
    case FP4LIN_ERR_VALUE: return "a number argument is NaN or out of range";
    case FP4LIN_ERR_OVERLAP: return "an output overlaps another one or an operand";
  }
  return "unknown status";
}

}  // extern "C"

namespace {

// The select's argument checks apart from the workspace.
fp4lin_status select_check(const void* A, fp4lin_dtype dt, int64_t M, int64_t K, int64_t lda,
                           double q, const float* tau, const fp4lin_coo& dA) {
  if (A == nullptr || tau == nullptr || dA.row == nullptr || dA.col == nullptr ||
      dA.val == nullptr || dA.row_ptr == nullptr)
    return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(M) || !ok_dim(K) || lda < K) return FP4LIN_ERR_SHAPE;
  const int64_t n = M * K;
  if (n >= kMaxCount) return FP4LIN_ERR_SHAPE;
  const int64_t k = fp4lin_quantile_rank(n, q);
  if (k < 0) return FP4LIN_ERR_QUANTILE;
  const int64_t cap = needed_capacity(n, k);
  if (cap >= kMaxDim) return FP4LIN_ERR_SHAPE;
  if (dA.capacity < cap) return FP4LIN_ERR_CAPACITY;
  return FP4LIN_OK;
}

// fp4lin_outlier_select; with quantized set, the forward path's token-wise
// quantization of A (Xq, sX) is done by the same kernels where the rows allow
// it, and *quantized says whether it was.
fp4lin::FrontArgs front_args(const void* A, fp4lin_dtype dt, bool mx, int64_t M, int64_t K,
                             int64_t lda, double q, float* tau, const fp4lin_coo& coo,
                             void* scratch, uint8_t* Aq, int64_t ldq, void* sA, const void* W,
                             int64_t N, int64_t ldw, uint8_t* Wq, void* sW, uint32_t* colmax) {
  fp4lin::FrontArgs f;
  f.A = A;
  f.bf16 = dt == FP4LIN_BF16;
  f.mx = mx;
  f.M = M;
  f.K = K;
  f.lda = lda;
  f.k = fp4lin_quantile_rank(M * K, q);
  f.tau = tau;
  f.capacity = coo.capacity;
  f.row = coo.row;
  f.col = coo.col;
  f.val = coo.val;
  f.row_ptr = coo.row_ptr;
  f.ws = scratch;
  f.Aq = Aq;
  f.ldq = ldq;
  f.sA = sA;
  f.W = W;
  f.N = N;
  f.ldw = ldw;
  f.Wq = Wq;
  f.sW = sW;
  f.colmax = colmax;
  return f;
}
fp4lin_status select_impl(const void* A, fp4lin_dtype dt, int64_t M, int64_t K, int64_t lda,
                          double q, float* tau, fp4lin_coo dA, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  if (ws == nullptr) return FP4LIN_ERR_NULL;
  const fp4lin_status c = select_check(A, dt, M, K, lda, q, tau, dA);
  if (c != FP4LIN_OK) return c;
  if (!aligned16(ws)) return FP4LIN_ERR_ALIGN;
  if (ws_bytes < select_ws(M, dt)) return FP4LIN_ERR_WORKSPACE;
  return launch_status(fp4lin::launch_outlier_select(
      A, dt == FP4LIN_BF16, M, K, lda, fp4lin_quantile_rank(M * K, q), tau, dA.capacity,
      dA.row, dA.col, dA.val, dA.row_ptr, ws, stream));
}

// ---- allocation-free select ---------------------------------------------------
// fp4lin_outlier_select_noalloc keeps the select's scratch (selection state,
// histograms, per-row counts) in this array: one copy per GPU the library
// runs on, held until the process ends. In host code its name is only a
// host-side stand-in; the device address of each GPU's copy is looked up once
// per device, with that device current, and only that address is used.
// None of the select's kernels relies on the scratch being cleared, so the
// contents a previous call left are harmless.
constexpr size_t kNoAllocScratchBytes = size_t(8) << 20;
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 256;
std::mutex g_scratch_mutex;
void* g_scratch_addr[kMaxDevices];

// This GPU's copy of the scratch: the device of `stream` (the current device
// for the null stream), looked up on the first call for that device.
hipError_t scratch_address(hipStream_t stream, void** out) {
  int dev = 0;
  hipError_t e = hipStreamGetDevice(stream, &dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (g_scratch_addr[dev] == nullptr) {
    int cur = 0;
    e = hipGetDevice(&cur);
    if (e != hipSuccess) return e;
    if (cur != dev) {
      e = hipSetDevice(dev);
      if (e != hipSuccess) return e;
    }
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (cur != dev) {
      const hipError_t back = hipSetDevice(cur);
      if (e == hipSuccess) e = back;
    }
    if (e != hipSuccess) return e;
    if (p == nullptr) return hipErrorInvalidSymbol;
    g_scratch_addr[dev] = p;
  }
  *out = g_scratch_addr[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

fp4lin_status fp4lin_outlier_select(const void* A, fp4lin_dtype dt, int64_t M, int64_t K,
                                    int64_t lda, double q, float* tau, fp4lin_coo dA, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  return select_impl(A, dt, M, K, lda, q, tau, dA, ws, ws_bytes, stream);
}

fp4lin_status fp4lin_outlier_select_noalloc(const void* A, fp4lin_dtype dt, int64_t M,
                                            int64_t K, int64_t lda, double q, float* tau,
                                            fp4lin_coo dA, hipStream_t stream) {
  const fp4lin_status c = select_check(A, dt, M, K, lda, q, tau, dA);
  if (c != FP4LIN_OK) return c;
  if (select_ws(M, dt) > kNoAllocScratchBytes) return FP4LIN_ERR_SCRATCH;
  void* ws = nullptr;
  const hipError_t e = scratch_address(stream, &ws);
  if (e != hipSuccess) return launch_status(e);
  return select_impl(A, dt, M, K, lda, q, tau, dA, ws, kNoAllocScratchBytes, stream);
}

fp4lin_status fp4lin_quantize_act(const void* X, fp4lin_dtype dt, int64_t M, int64_t K,
                                  int64_t ldx, const float* tau, uint8_t* Xq, float* sX,
                                  hipStream_t stream) {
  if (X == nullptr || Xq == nullptr || sX == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(M) || !ok_dim(K) || ldx < K) return FP4LIN_ERR_SHAPE;
  if (!aligned16(Xq)) return FP4LIN_ERR_ALIGN;
  return launch_status(fp4lin::launch_quantize_rows(X, dt == FP4LIN_BF16, M, K, ldx, tau, Xq,
                                                    fp4lin_packed_ld(K), sX, stream));
}

fp4lin_status fp4lin_quantize_weight(const void* W, fp4lin_dtype dt, int64_t K, int64_t N,
                                     int64_t ldw, uint8_t* Wq, float* sW, void* ws,
                                     size_t ws_bytes, hipStream_t stream) {
  if (W == nullptr || Wq == nullptr || sW == nullptr || ws == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(K) || !ok_dim(N) || ldw < N || K > kMaxColK || !col_grids_fit(K, N))
    return FP4LIN_ERR_SHAPE;
  if (!aligned16(Wq) || !aligned16(ws)) return FP4LIN_ERR_ALIGN;
  if (ws_bytes < weight_ws(N)) return FP4LIN_ERR_WORKSPACE;
  return launch_status(fp4lin::launch_quantize_weight(W, dt == FP4LIN_BF16, K, N, ldw, Wq,
                                                      fp4lin_packed_ld(K), sW, ws, stream));
}

fp4lin_status fp4lin_gemm(const uint8_t* Aq, const float* sA, const uint8_t* Bq, const float* sB,
                          int64_t M, int64_t N, int64_t K, const fp4lin_coo* dA, const void* W,
                          fp4lin_dtype wdt, int64_t ldw, float* Y, int64_t ldy,
                          hipStream_t stream) {
  if (Aq == nullptr || sA == nullptr || Bq == nullptr || sB == nullptr || Y == nullptr)
    return FP4LIN_ERR_NULL;
  if (!ok_dim(M) || !ok_dim(N) || !ok_dim(K) || ldy < N) return FP4LIN_ERR_SHAPE;
  fp4lin::SparseArgs sp{nullptr, nullptr, nullptr, nullptr, false, 0, 0, 0};
  if (dA != nullptr) {
    if (dA->row_ptr == nullptr || dA->col == nullptr || dA->val == nullptr || W == nullptr)
      return FP4LIN_ERR_NULL;
    if (bad_dtype(wdt)) return FP4LIN_ERR_DTYPE;
    if (ldw < N || !weight_addressable(K, ldw, wdt)) return FP4LIN_ERR_SHAPE;
    sp = fp4lin::SparseArgs{dA->row_ptr, dA->col, dA->val, W, wdt == FP4LIN_BF16, ldw, K,
                            dA->capacity};
  }
  // packed operands are addressed with 32-bit byte offsets
  const int64_t ldq = fp4lin_packed_ld(K);
  if ((M + 1) * ldq >= kMaxDim || (N + 1) * ldq >= kMaxDim) return FP4LIN_ERR_SHAPE;
  if (!aligned16(Aq) || !aligned16(Bq)) return FP4LIN_ERR_ALIGN;
  return launch_status(
      fp4lin::launch_fp4_gemm(Aq, sA, Bq, sB, M, N, fp4lin_packed_ld(K), sp, Y, ldy, stream));
}

fp4lin_status fp4lin_sparse_add(const fp4lin_coo* dA, const void* W, fp4lin_dtype wdt,
                                int64_t K, int64_t ldw, int64_t M, int64_t N, float* Y,
                                int64_t ldy, hipStream_t stream) {
  if (dA == nullptr || dA->row_ptr == nullptr || dA->col == nullptr || dA->val == nullptr ||
      W == nullptr || Y == nullptr)
    return FP4LIN_ERR_NULL;
  if (bad_dtype(wdt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(M) || !ok_dim(N) || !ok_dim(K) || ldw < N || ldy < N ||
      !weight_addressable(K, ldw, wdt))
    return FP4LIN_ERR_SHAPE;
  const fp4lin::SparseArgs sp{dA->row_ptr, dA->col, dA->val, W, wdt == FP4LIN_BF16,
                              ldw,         K,       dA->capacity};
  return launch_status(fp4lin::launch_sparse_add(sp, M, N, Y, ldy, stream));
}

int64_t fp4lin_mx_scales_ld(int64_t L) {
  if (L < 1) return -1;
  return fp4lin_packed_ld(L) / 16;
}

fp4lin_status fp4lin_quantize_act_mx(const void* X, fp4lin_dtype dt, int64_t M, int64_t K,
                                     int64_t ldx, const float* tau, uint8_t* Xq, uint8_t* Xs,
                                     hipStream_t stream) {
  if (X == nullptr || Xq == nullptr || Xs == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(M) || !ok_dim(K) || ldx < K) return FP4LIN_ERR_SHAPE;
  if (!aligned16(Xq) || !aligned16(Xs)) return FP4LIN_ERR_ALIGN;
  return launch_status(fp4lin::launch_quantize_rows_mx(X, dt == FP4LIN_BF16, M, K, ldx, tau, Xq,
                                                       fp4lin_packed_ld(K), Xs, stream));
}

fp4lin_status fp4lin_quantize_weight_mx(const void* W, fp4lin_dtype dt, int64_t K, int64_t N,
                                        int64_t ldw, uint8_t* Wq, uint8_t* Ws,
                                        hipStream_t stream) {
  if (W == nullptr || Wq == nullptr || Ws == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(K) || !ok_dim(N) || ldw < N || K > kMaxColK || !col_grids_fit(K, N))
    return FP4LIN_ERR_SHAPE;
  if (!aligned16(Wq) || !aligned16(Ws)) return FP4LIN_ERR_ALIGN;
  return launch_status(fp4lin::launch_quantize_cols_mx(W, dt == FP4LIN_BF16, K, N, ldw, Wq,
                                                       fp4lin_packed_ld(K), Ws, stream));
}

fp4lin_status fp4lin_gemm_mx(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                             const uint8_t* Bs, int64_t M, int64_t N, int64_t K,
                             const fp4lin_coo* dA, const void* W, fp4lin_dtype wdt,
                             int64_t ldw, float* Y, int64_t ldy, hipStream_t stream) {
  if (Aq == nullptr || As == nullptr || Bq == nullptr || Bs == nullptr || Y == nullptr)
    return FP4LIN_ERR_NULL;
  if (!ok_dim(M) || !ok_dim(N) || !ok_dim(K) || ldy < N) return FP4LIN_ERR_SHAPE;
  fp4lin::SparseArgs sp{nullptr, nullptr, nullptr, nullptr, false, 0, 0, 0};
  if (dA != nullptr) {
    if (dA->row_ptr == nullptr || dA->col == nullptr || dA->val == nullptr || W == nullptr)
      return FP4LIN_ERR_NULL;
    if (bad_dtype(wdt)) return FP4LIN_ERR_DTYPE;
    if (ldw < N || !weight_addressable(K, ldw, wdt)) return FP4LIN_ERR_SHAPE;
    sp = fp4lin::SparseArgs{dA->row_ptr, dA->col, dA->val, W, wdt == FP4LIN_BF16, ldw, K,
                            dA->capacity};
  }
  // packed operands and scale rows are addressed with 32-bit byte offsets
  const int64_t ldq = fp4lin_packed_ld(K);
  if ((M + 1) * ldq >= kMaxDim || (N + 1) * ldq >= kMaxDim) return FP4LIN_ERR_SHAPE;
  if (!aligned16(Aq) || !aligned16(Bq) || !aligned16(As) || !aligned16(Bs))
    return FP4LIN_ERR_ALIGN;
  return launch_status(fp4lin::launch_fp4_gemm_mx(Aq, As, Bq, Bs, M, N, ldq, sp, Y, ldy, stream));
}

fp4lin_status fp4lin_forward(const void* A, const void* W, fp4lin_dtype dt, int64_t M, int64_t K,
                             int64_t N, int64_t lda, int64_t ldw, double q, float* Y, int64_t ldy,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  if (A == nullptr || W == nullptr || Y == nullptr || ws == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(M) || !ok_dim(K) || !ok_dim(N) || lda < K || ldw < N || ldy < N)
    return FP4LIN_ERR_SHAPE;
  fp4lin_forward_offsets o;
  const fp4lin_status ls = fp4lin_forward_layout(M, K, N, dt, q, &o);
  if (ls != FP4LIN_OK) return ls;
  if (!aligned16(ws)) return FP4LIN_ERR_ALIGN;
  if (ws_bytes < o.total) return FP4LIN_ERR_WORKSPACE;
  // the limits of the GEMM and of W's quantizer, checked before anything is
  // enqueued
  const int64_t ldq = fp4lin_packed_ld(K);
  if ((M + 1) * ldq >= kMaxDim || (N + 1) * ldq >= kMaxDim || !weight_addressable(K, ldw, dt) ||
      K > kMaxColK)
    return FP4LIN_ERR_SHAPE;
  char* base = static_cast<char*>(ws);
  float* tau = reinterpret_cast<float*>(base + o.tau);
  fp4lin_coo coo;
  coo.row = reinterpret_cast<int32_t*>(base + o.coo_row);
  coo.col = reinterpret_cast<int32_t*>(base + o.coo_col);
  coo.val = reinterpret_cast<float*>(base + o.coo_val);
  coo.row_ptr = reinterpret_cast<int32_t*>(base + o.row_ptr);
  coo.capacity = o.capacity;
  uint8_t* Aq = reinterpret_cast<uint8_t*>(base + o.Aq);
  float* sA = reinterpret_cast<float*>(base + o.sA);
  uint8_t* Wq = reinterpret_cast<uint8_t*>(base + o.Wq);
  float* sW = reinterpret_cast<float*>(base + o.sW);
  void* scratch = base + o.scratch;
  // select, quantization of A (in the select's compaction) and of W (in the
  // select's row launches); W's column maxima follow the select's workspace
  const fp4lin::FrontArgs f = front_args(A, dt, false, M, K, lda, q, tau, coo, scratch, Aq, ldq, sA,
                                         W, N, ldw, Wq, sW,
                                         reinterpret_cast<uint32_t*>(static_cast<char*>(scratch) +
                                                                     select_ws(M, dt)));
  const fp4lin_status s = launch_status(fp4lin::launch_forward_front(f, stream));
  if (s != FP4LIN_OK) return s;
  return fp4lin_gemm(Aq, sA, Wq, sW, M, N, K, &coo, W, dt, ldw, Y, ldy, stream);
}

fp4lin_status fp4lin_forward_mx(const void* A, const void* W, fp4lin_dtype dt, int64_t M,
                                int64_t K, int64_t N, int64_t lda, int64_t ldw, double q,
                                float* Y, int64_t ldy, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  if (A == nullptr || W == nullptr || Y == nullptr || ws == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  if (!ok_dim(M) || !ok_dim(K) || !ok_dim(N) || lda < K || ldw < N || ldy < N)
    return FP4LIN_ERR_SHAPE;
  fp4lin_forward_offsets o;
  const fp4lin_status ls = fp4lin_forward_layout_mx(M, K, N, dt, q, &o);
  if (ls != FP4LIN_OK) return ls;
  if (!aligned16(ws)) return FP4LIN_ERR_ALIGN;
  if (ws_bytes < o.total) return FP4LIN_ERR_WORKSPACE;
  // the limits of the GEMM and of W's quantizer, checked before anything is
  // enqueued
  const int64_t ldq = fp4lin_packed_ld(K);
  if ((M + 1) * ldq >= kMaxDim || (N + 1) * ldq >= kMaxDim || !weight_addressable(K, ldw, dt) ||
      K > kMaxColK)
    return FP4LIN_ERR_SHAPE;
  char* base = static_cast<char*>(ws);
  float* tau = reinterpret_cast<float*>(base + o.tau);
  fp4lin_coo coo;
  coo.row = reinterpret_cast<int32_t*>(base + o.coo_row);
  coo.col = reinterpret_cast<int32_t*>(base + o.coo_col);
  coo.val = reinterpret_cast<float*>(base + o.coo_val);
  coo.row_ptr = reinterpret_cast<int32_t*>(base + o.row_ptr);
  coo.capacity = o.capacity;
  uint8_t* Aq = reinterpret_cast<uint8_t*>(base + o.Aq);
  uint8_t* As = reinterpret_cast<uint8_t*>(base + o.sA);
  uint8_t* Wq = reinterpret_cast<uint8_t*>(base + o.Wq);
  uint8_t* Ws = reinterpret_cast<uint8_t*>(base + o.sW);
  void* scratch = base + o.scratch;
  // select, micro-scaled quantization of A (in the select's compaction) and
  // of W (in the select's row-count launch)
  const fp4lin::FrontArgs f = front_args(A, dt, true, M, K, lda, q, tau, coo, scratch, Aq, ldq, As,
                                         W, N, ldw, Wq, Ws, nullptr);
  const fp4lin_status s = launch_status(fp4lin::launch_forward_front(f, stream));
  if (s != FP4LIN_OK) return s;
  return fp4lin_gemm_mx(Aq, As, Wq, Ws, M, N, K, &coo, W, dt, ldw, Y, ldy, stream);
}

}  // extern "C"

// ---- products grouped by expert -------------------------------------------------
namespace {

constexpr int64_t kMaxExperts = 65534;  // experts index a grid dimension, one group more

bool ok_rows(int64_t M) { return M >= 0 && M < kMaxDim; }

// Sizes that every pass checks; the offsets of a pass's operands besides.
fp4lin_status experts_sizes(int64_t E, int64_t M, int64_t K, int64_t N) {
  if (E < 1 || E > kMaxExperts || !ok_rows(M) || !ok_dim(K) || !ok_dim(N)) return FP4LIN_ERR_SHAPE;
  return FP4LIN_OK;
}

// Packed rows of ldq bytes that one resource covers, and the scales of `all`
// packed rows of L codes.
bool packed_fits(int64_t rows, int64_t ldq) { return (rows + 1) * ldq < kMaxDim; }
bool scales_fit(int64_t all, int64_t L) {
  return double(all) * double(fp4lin_mx_scales_ld(L)) < double(kMaxDim);
}

// Workgroups of the tiled products (at the finest 128 x 256 tiles) and of the
// quantizers fit a grid.
bool tiles_fit(double rows, double groups, double cols) {
  return (rows / 128 + groups + 1) * (cols / 256 + 1) < double(kMaxDim);
}

// Reduction along L of M rows against E * n rows of weights (forward: L = K,
// n = N; dgrad: L = N, n = K).
fp4lin_status experts_rows_fit(int64_t E, int64_t M, int64_t L, int64_t n) {
  const int64_t ldq = fp4lin_packed_ld(L);
  if (!packed_fits(M, ldq) || !packed_fits(n, ldq) || !scales_fit(E * n, L) || !scales_fit(M, L) ||
      L > kMaxColK || !tiles_fit(double(M), double(E), double(n)))
    return FP4LIN_ERR_SHAPE;
  return FP4LIN_OK;
}

fp4lin_status experts_cols_fit(int64_t E, int64_t M, int64_t K, int64_t N) {
  const int64_t steps = fp4lin::experts_steps(E, M);
  const int64_t most = K > N ? K : N;
  if (steps > 65535 || double(most) * double(steps + 1) * 64 >= double(kMaxDim) ||
      double(E) * (double(K) / 128 + 1) * (double(N) / 256 + 1) >= double(kMaxDim))
    return FP4LIN_ERR_SHAPE;
  return FP4LIN_OK;
}

// Where a pass keeps its two quantized operands in the workspace.
struct ExpertsLayout {
  size_t Aq, As, Bq, Bs, total;
};

fp4lin_status experts_layout(fp4lin_experts_pass pass, int64_t E, int64_t M, int64_t K, int64_t N,
                             ExpertsLayout* out) {
  fp4lin_status s = experts_sizes(E, M, K, N);
  if (s != FP4LIN_OK) return s;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  ExpertsLayout o{};
  if (pass == FP4LIN_EXPERTS_WGRAD) {
    s = experts_cols_fit(E, M, K, N);
    if (s != FP4LIN_OK) return s;
    const size_t steps = size_t(fp4lin::experts_steps(E, M));
    o.Aq = take(size_t(K) * steps * 64);
    o.As = take(size_t(K) * steps * 4);
    o.Bq = take(size_t(N) * steps * 64);
    o.Bs = take(size_t(N) * steps * 4);
  } else if (pass == FP4LIN_EXPERTS_FORWARD || pass == FP4LIN_EXPERTS_DGRAD ||
             pass == FP4LIN_EXPERTS_APPLY) {
    const int64_t L = pass == FP4LIN_EXPERTS_DGRAD ? N : K;
    const int64_t n = pass == FP4LIN_EXPERTS_DGRAD ? K : N;
    s = experts_rows_fit(E, M, L, n);
    if (s != FP4LIN_OK) return s;
    const size_t ldq = size_t(fp4lin_packed_ld(L)), lds = size_t(fp4lin_mx_scales_ld(L));
    o.Aq = take(size_t(M) * ldq);
    o.As = take(size_t(M) * lds);
    if (pass != FP4LIN_EXPERTS_APPLY) {
      o.Bq = take(size_t(E) * size_t(n) * ldq);
      o.Bs = take(size_t(E) * size_t(n) * lds);
    }
  } else {
    return FP4LIN_ERR_SHAPE;
  }
  o.total = off > 256 ? off : 256;
  *out = o;
  return FP4LIN_OK;
}

fp4lin_status experts_workspace(fp4lin_experts_pass pass, int64_t E, int64_t M, int64_t K,
                                int64_t N, const void* ws, size_t ws_bytes, ExpertsLayout* out) {
  const fp4lin_status s = experts_layout(pass, E, M, K, N, out);
  if (s != FP4LIN_OK) return s;
  if (ws == nullptr) return FP4LIN_ERR_NULL;
  if (!aligned16(ws)) return FP4LIN_ERR_ALIGN;
  return ws_bytes < out->total ? FP4LIN_ERR_WORKSPACE : FP4LIN_OK;
}

}  // namespace

extern "C" {

size_t fp4lin_experts_workspace_bytes(fp4lin_experts_pass pass, int64_t E, int64_t M, int64_t K,
                                      int64_t N) {
  ExpertsLayout o;
  return experts_layout(pass, E, M, K, N, &o) == FP4LIN_OK ? o.total : 0;
}

fp4lin_status fp4lin_experts_quantize_weight_mx(const void* W, fp4lin_dtype dt, int64_t E,
                                                int64_t K, int64_t N, int64_t ldw, uint8_t* Wq,
                                                uint8_t* Ws, hipStream_t stream) {
  if (W == nullptr || Wq == nullptr || Ws == nullptr) return FP4LIN_ERR_NULL;
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  fp4lin_status s = experts_sizes(E, 0, K, N);
  if (s == FP4LIN_OK) s = experts_rows_fit(E, 0, K, N);
  if (s != FP4LIN_OK) return s;
  if (ldw < N) return FP4LIN_ERR_SHAPE;
  if (!aligned16(Wq) || !aligned16(Ws)) return FP4LIN_ERR_ALIGN;
  return launch_status(fp4lin::launch_experts_quantize_weight_mx(
      W, dt == FP4LIN_BF16, E, K, N, ldw, Wq, fp4lin_packed_ld(K), Ws, stream));
}

fp4lin_status fp4lin_experts_forward_mx(const void* A, const void* W, fp4lin_dtype dt,
                                        const int32_t* row_end, int64_t E, int64_t M, int64_t K,
                                        int64_t N, int64_t lda, int64_t ldw, void* Y,
                                        fp4lin_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes,
                                        hipStream_t stream) {
  if (W == nullptr || row_end == nullptr || (M != 0 && (A == nullptr || Y == nullptr)))
    return FP4LIN_ERR_NULL;
  if (bad_dtype(dt) || bad_dtype(ydt)) return FP4LIN_ERR_DTYPE;
  ExpertsLayout o;
  fp4lin_status s = experts_workspace(FP4LIN_EXPERTS_FORWARD, E, M, K, N, ws, ws_bytes, &o);
  if (s != FP4LIN_OK) return s;
  if (lda < K || ldw < N || ldy < N) return FP4LIN_ERR_SHAPE;
  if (M == 0) return FP4LIN_OK;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  const int64_t ldq = fp4lin_packed_ld(K);
  s = launch_status(fp4lin::launch_experts_quantize_forward(A, W, dt == FP4LIN_BF16, E, M, K, N, lda,
                                                            ldw, base + o.Aq, base + o.As,
                                                            base + o.Bq, base + o.Bs, stream));
  if (s != FP4LIN_OK) return s;
  return launch_status(fp4lin::launch_experts_rows(base + o.Aq, base + o.As, base + o.Bq,
                                                   base + o.Bs, row_end, E, M, N, ldq, false, Y,
                                                   ydt == FP4LIN_BF16, ldy, stream));
}

fp4lin_status fp4lin_experts_apply_mx(const void* A, fp4lin_dtype dt, const uint8_t* Wq,
                                      const uint8_t* Ws, const int32_t* row_end, int64_t E,
                                      int64_t M, int64_t K, int64_t N, int64_t lda, void* Y,
                                      fp4lin_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes,
                                      hipStream_t stream) {
  if (Wq == nullptr || Ws == nullptr || row_end == nullptr ||
      (M != 0 && (A == nullptr || Y == nullptr)))
    return FP4LIN_ERR_NULL;
  if (bad_dtype(dt) || bad_dtype(ydt)) return FP4LIN_ERR_DTYPE;
  ExpertsLayout o;
  fp4lin_status s = experts_workspace(FP4LIN_EXPERTS_APPLY, E, M, K, N, ws, ws_bytes, &o);
  if (s != FP4LIN_OK) return s;
  if (lda < K || ldy < N) return FP4LIN_ERR_SHAPE;
  if (!aligned16(Wq) || !aligned16(Ws)) return FP4LIN_ERR_ALIGN;
  if (M == 0) return FP4LIN_OK;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  const int64_t ldq = fp4lin_packed_ld(K);
  if (fp4lin::experts_fused(M, K))
    return launch_status(fp4lin::launch_experts_fused(A, dt == FP4LIN_BF16, lda, Wq, Ws, row_end, E,
                                                      M, K, N, ldq, Y, ydt == FP4LIN_BF16, ldy,
                                                      stream));
  s = launch_status(fp4lin::launch_experts_quantize_rows(A, dt == FP4LIN_BF16, M, K, lda,
                                                         base + o.Aq, base + o.As, stream));
  if (s != FP4LIN_OK) return s;
  return launch_status(fp4lin::launch_experts_rows(base + o.Aq, base + o.As, Wq, Ws, row_end, E, M,
                                                   N, ldq, true, Y, ydt == FP4LIN_BF16, ldy,
                                                   stream));
}

fp4lin_status fp4lin_experts_dgrad_mx(const void* dY, const void* W, fp4lin_dtype dt,
                                      const int32_t* row_end, int64_t E, int64_t M, int64_t K,
                                      int64_t N, int64_t lddy, int64_t ldw, void* dX,
                                      fp4lin_dtype xdt, int64_t lddx, void* ws, size_t ws_bytes,
                                      hipStream_t stream) {
  if (W == nullptr || row_end == nullptr || (M != 0 && (dY == nullptr || dX == nullptr)))
    return FP4LIN_ERR_NULL;
  if (bad_dtype(dt) || bad_dtype(xdt)) return FP4LIN_ERR_DTYPE;
  ExpertsLayout o;
  fp4lin_status s = experts_workspace(FP4LIN_EXPERTS_DGRAD, E, M, K, N, ws, ws_bytes, &o);
  if (s != FP4LIN_OK) return s;
  if (lddy < N || ldw < N || lddx < K) return FP4LIN_ERR_SHAPE;
  if (M == 0) return FP4LIN_OK;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  const int64_t ldq = fp4lin_packed_ld(N);
  s = launch_status(fp4lin::launch_experts_quantize_dgrad(dY, W, dt == FP4LIN_BF16, E, M, K, N, lddy,
                                                          ldw, base + o.Aq, base + o.As,
                                                          base + o.Bq, base + o.Bs, stream));
  if (s != FP4LIN_OK) return s;
  return launch_status(fp4lin::launch_experts_rows(base + o.Aq, base + o.As, base + o.Bq,
                                                   base + o.Bs, row_end, E, M, K, ldq, false, dX,
                                                   xdt == FP4LIN_BF16, lddx, stream));
}

fp4lin_status fp4lin_experts_wgrad_mx(const void* A, const void* dY, fp4lin_dtype dt,
                                      const int32_t* row_end, int64_t E, int64_t M, int64_t K,
                                      int64_t N, int64_t lda, int64_t lddy, void* dW,
                                      fp4lin_dtype wdt, int64_t lddw, void* ws, size_t ws_bytes,
                                      hipStream_t stream) {
  if (dW == nullptr || row_end == nullptr || (M != 0 && (A == nullptr || dY == nullptr)))
    return FP4LIN_ERR_NULL;
  if (bad_dtype(dt) || bad_dtype(wdt)) return FP4LIN_ERR_DTYPE;
  ExpertsLayout o;
  fp4lin_status s = experts_workspace(FP4LIN_EXPERTS_WGRAD, E, M, K, N, ws, ws_bytes, &o);
  if (s != FP4LIN_OK) return s;
  if (lda < K || lddy < N || lddw < N) return FP4LIN_ERR_SHAPE;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  s = launch_status(fp4lin::launch_experts_quantize_wgrad(A, dY, dt == FP4LIN_BF16, row_end, E, M, K,
                                                          N, lda, lddy, base + o.Aq, base + o.As,
                                                          base + o.Bq, base + o.Bs, stream));
  if (s != FP4LIN_OK) return s;
  return launch_status(fp4lin::launch_experts_wgrad(base + o.Aq, base + o.As, base + o.Bq,
                                                    base + o.Bs, row_end, E, M, K, N, dW,
                                                    wdt == FP4LIN_BF16, lddw, stream));
}

}  // extern "C"

// ---- head loss ------------------------------------------------------------------
namespace {

struct HeadLayout {
  fp4lin::HeadPlan plan;
  size_t x, w, part, tlogit, G, acc, top, total;
};

// Sizes and strides that both calls check, and where they keep what they keep.
fp4lin_status head_layout(fp4lin_dtype dt, fp4lin_head_layout layout, int64_t T, int64_t H,
                          int64_t V, int64_t ldx, int64_t ldw, bool backward, HeadLayout* out) {
  if (bad_dtype(dt)) return FP4LIN_ERR_DTYPE;
  const bool by_vocab = layout == FP4LIN_HEAD_VOCAB_MAJOR;
  if (!by_vocab && layout != FP4LIN_HEAD_HIDDEN_MAJOR) return FP4LIN_ERR_SHAPE;
  const int64_t esz = dt == FP4LIN_BF16 ? 2 : 4;
  const int64_t most = kMaxDim / 256 / esz - 16;  // of a leading dimension
  if (!ok_rows(T) || !ok_dim(H) || !ok_dim(V) || ldx < H || ldw < (by_vocab ? H : V))
    return FP4LIN_ERR_SHAPE;
  if (ldx > most || ldw > most || H > most || V > most || T > (int64_t(1) << 22))
    return FP4LIN_ERR_SHAPE;
  // tiles index a grid of at most 2^31 - 1 workgroups
  if ((double(T) / 64 + 1) * (double(V) / 128 + 1) >= double(kMaxDim)) return FP4LIN_ERR_SHAPE;
  HeadLayout o{};
  o.plan = fp4lin::head_plan(dt == FP4LIN_BF16, backward, T, H, V, by_vocab, ldx, ldw);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  o.x = take(size_t(o.plan.x_bytes));
  o.w = take(size_t(o.plan.w_bytes));
  if (backward) {
    o.G = take(size_t(T) * size_t(o.plan.ldg) * size_t(esz));
    o.acc = take(size_t(T) * size_t(o.plan.ldp) * size_t(o.plan.slices) * 4);
    o.top = take(4);
  } else {
    o.part = take(size_t(T) * size_t(o.plan.parts) * 8);
    o.tlogit = take(size_t(T) * 4);
  }
  o.total = off > 256 ? off : 256;
  *out = o;
  return FP4LIN_OK;
}

fp4lin_status head_call(const void* X, const void* W, fp4lin_dtype dt, fp4lin_head_layout layout,
                        const int32_t* target, int64_t T, int64_t H, int64_t V, int64_t ldx,
                        int64_t ldw, void* ws, size_t ws_bytes, bool backward, HeadLayout* o,
                        fp4lin::HeadCall* c) {
  const fp4lin_status s = head_layout(dt, layout, T, H, V, ldx, ldw, backward, o);
  if (s != FP4LIN_OK) return s;
  if (ws == nullptr) return FP4LIN_ERR_NULL;
  if (!aligned16(ws) || !aligned16(X) || !aligned16(W)) return FP4LIN_ERR_ALIGN;
  if (ws_bytes < o->total) return FP4LIN_ERR_WORKSPACE;
  char* const base = static_cast<char*>(ws);
  *c = fp4lin::HeadCall{};
  c->X = X;
  c->W = W;
  c->T = T;
  c->H = H;
  c->V = V;
  c->ldx = ldx;
  c->ldw = ldw;
  c->by_vocab = layout == FP4LIN_HEAD_VOCAB_MAJOR;
  c->target = target;
  c->packed_x = base + o->x;
  c->packed_w = base + o->w;
  c->part = base + o->part;
  c->tlogit = reinterpret_cast<float*>(base + o->tlogit);
  c->G = base + o->G;
  c->acc = reinterpret_cast<float*>(base + o->acc);
  c->top = reinterpret_cast<float*>(base + o->top);
  return FP4LIN_OK;
}

}  // namespace

extern "C" {

size_t fp4lin_head_loss_workspace_bytes(fp4lin_dtype dt, fp4lin_head_layout layout, int64_t T,
                                        int64_t H, int64_t V, int64_t ldx, int64_t ldw) {
  HeadLayout o;
  return head_layout(dt, layout, T, H, V, ldx, ldw, false, &o) == FP4LIN_OK ? o.total : 0;
}

size_t fp4lin_head_loss_backward_workspace_bytes(fp4lin_dtype dt, fp4lin_head_layout layout,
                                                 int64_t T, int64_t H, int64_t V, int64_t ldx,
                                                 int64_t ldw) {
  HeadLayout o;
  return head_layout(dt, layout, T, H, V, ldx, ldw, true, &o) == FP4LIN_OK ? o.total : 0;
}

fp4lin_status fp4lin_head_loss(const void* X, const void* W, fp4lin_dtype dt,
                               fp4lin_head_layout layout, const int32_t* target, int64_t T,
                               int64_t H, int64_t V, int64_t ldx, int64_t ldw, float* loss,
                               float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (W == nullptr ||
      (T != 0 && (X == nullptr || target == nullptr || loss == nullptr || lse == nullptr)))
    return FP4LIN_ERR_NULL;
  HeadLayout o;
  fp4lin::HeadCall c;
  const fp4lin_status s =
      head_call(X, W, dt, layout, target, T, H, V, ldx, ldw, ws, ws_bytes, false, &o, &c);
  if (s != FP4LIN_OK || T == 0) return s;
  c.loss = loss;
  c.lse_out = lse;
  return launch_status(fp4lin::launch_head_loss(c, dt == FP4LIN_BF16, o.plan, stream));
}

fp4lin_status fp4lin_head_loss_backward(const void* X, const void* W, fp4lin_dtype dt,
                                        fp4lin_head_layout layout, const int32_t* target,
                                        const float* lse, const float* dloss, int64_t T, int64_t H,
                                        int64_t V, int64_t ldx, int64_t ldw, void* dX, int64_t lddx,
                                        void* dW, int64_t lddw, void* ws, size_t ws_bytes,
                                        hipStream_t stream) {
  if (W == nullptr || dW == nullptr ||
      (T != 0 && (X == nullptr || target == nullptr || lse == nullptr || dloss == nullptr ||
                  dX == nullptr)))
    return FP4LIN_ERR_NULL;
  HeadLayout o;
  fp4lin::HeadCall c;
  const fp4lin_status s =
      head_call(X, W, dt, layout, target, T, H, V, ldx, ldw, ws, ws_bytes, true, &o, &c);
  if (s != FP4LIN_OK) return s;
  if (lddx < H || lddw < (c.by_vocab ? H : V)) return FP4LIN_ERR_SHAPE;
  c.lse = lse;
  c.dloss = dloss;
  c.dX = dX;
  c.dW = dW;
  c.lddx = lddx;
  c.lddw = lddw;
  return launch_status(fp4lin::launch_head_loss_backward(c, dt == FP4LIN_BF16, o.plan, stream));
}

}  // extern "C"

// ---- gradient norm and clipping ---------------------------------------------------
namespace {

constexpr int64_t kMaxElements = int64_t(1) << 46;

size_t clip_ws(int64_t count, int64_t elements) {
  return round_up(16 + size_t(fp4lin::clip_parts(count, elements)) * 8, 256);
}

// Whether memory that one workgroup writes is read or written by another tensor's:
// an output over another output or over a gradient not its own. (Gradients that are
// only read may overlap.) Sorted spans, kBlock tensors at a time on the stack; of more,
// every two blocks together. 42 tensors: below 1 us.
constexpr int64_t kBlock = 512;
struct Span {
  uintptr_t begin, end;
  bool written;
};

int spans_of(const fp4lin_grad* grads, int64_t count, int64_t block, Span* s) {
  int n = 0;
  const int64_t last = std::min(count, (block + 1) * kBlock);
  for (int64_t i = block * kBlock; i < last; ++i) {
    const fp4lin_grad& x = grads[i];
    if (x.n == 0) continue;
    const uintptr_t bytes = uintptr_t(x.n) * (x.dt == FP4LIN_BF16 ? 2 : 4);
    const uintptr_t out = reinterpret_cast<uintptr_t>(x.out), g = reinterpret_cast<uintptr_t>(x.g);
    s[n++] = Span{out, out + bytes, true};
    if (g != out) s[n++] = Span{g, g + bytes, false};
  }
  return n;
}

bool spans_meet(Span* s, int n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t read = 0, written = 0;  // ends of what came before
  for (int i = 0; i < n; ++i) {
    if (s[i].begin < written || (s[i].written && s[i].begin < read)) return true;
    uintptr_t& end = s[i].written ? written : read;
    end = std::max(end, s[i].end);
  }
  return false;
}

bool outputs_overlap(const fp4lin_grad* grads, int64_t count) {
  Span s[4 * kBlock];
  const int64_t blocks = (count + kBlock - 1) / kBlock;
  if (blocks <= 1) return spans_meet(s, spans_of(grads, count, 0, s));
  for (int64_t i = 0; i < blocks; ++i)
    for (int64_t j = i + 1; j < blocks; ++j) {
      const int n = spans_of(grads, count, i, s);
      if (spans_meet(s, n + spans_of(grads, count, j, s + n))) return true;
    }
  return false;
}

fp4lin_status clip_impl(const fp4lin_grad* grads, int64_t count, bool clip, double max_norm,
                        float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (norm == nullptr || ws == nullptr || (count > 0 && grads == nullptr)) return FP4LIN_ERR_NULL;
  if (count < 0 || count >= kMaxDim) return FP4LIN_ERR_SHAPE;
  int64_t elements = 0;
  for (int64_t i = 0; i < count; ++i) {
    const fp4lin_grad& x = grads[i];
    if (x.n < 0 || x.n > kMaxElements) return FP4LIN_ERR_SHAPE;
    if (bad_dtype(x.dt)) return FP4LIN_ERR_DTYPE;
    if (x.n > 0 && (x.g == nullptr || (clip && x.out == nullptr))) return FP4LIN_ERR_NULL;
    // elements at their own alignment
    const uintptr_t low = x.dt == FP4LIN_BF16 ? 1 : 3;
    if (x.n > 0 && ((reinterpret_cast<uintptr_t>(x.g) & low) != 0 ||
                    (clip && (reinterpret_cast<uintptr_t>(x.out) & low) != 0)))
      return FP4LIN_ERR_ALIGN;
    elements += x.n;
    if (elements > kMaxElements) return FP4LIN_ERR_SHAPE;
  }
  if (clip && !(max_norm >= 0.0)) return FP4LIN_ERR_VALUE;
  if (!aligned16(ws)) return FP4LIN_ERR_ALIGN;
  if (clip && outputs_overlap(grads, count)) return FP4LIN_ERR_OVERLAP;
  if (ws_bytes < clip_ws(count, elements)) return FP4LIN_ERR_WORKSPACE;
  return launch_status(
      fp4lin::launch_clip(grads, count, elements, clip, float(max_norm), norm, ws, stream));
}

}  // namespace

extern "C" {

size_t fp4lin_clip_workspace_bytes(int64_t count, int64_t elements) {
  if (count < 0 || count >= kMaxDim || elements < 0 || elements > kMaxElements) return 0;
  return clip_ws(count, elements);
}

fp4lin_status fp4lin_grad_norm(const fp4lin_grad* grads, int64_t count, float* norm, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  return clip_impl(grads, count, false, 0.0, norm, ws, ws_bytes, stream);
}

fp4lin_status fp4lin_clip_grads(const fp4lin_grad* grads, int64_t count, double max_norm,
                                float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  return clip_impl(grads, count, true, max_norm, norm, ws, ws_bytes, stream);
}

}  // extern "C"
