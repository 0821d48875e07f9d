// Global 2-norm of many tensors and clipping by it.
//
//   norm = sqrt(sum over all elements of all tensors of g^2)
//   out  = g * c,  c = min(1, max_norm / (norm + 1e-6))
//
// The tensors' addresses, sizes and types travel in the kernel arguments, up to
// kBatch tensors a launch, so a call needs no device copy of the list and can be
// captured. Every tensor is cut in chunks of whole 16-byte groups, one workgroup
// each; the chunk length follows from the total size so that the chunks of all
// tensors fill the GPU without being many. A workgroup sums its squares in
// double (the square of a float is exact there and cannot overflow) and writes
// one partial sum; the sums are then added in a fixed order, so the norm does not
// depend on timing. With one batch of tensors every workgroup of the clipping
// kernel adds the few partial sums itself, which saves a launch; with more, one
// workgroup adds them once.
//
// Bound by memory: each gradient is read for the norm and once more for the
// clipping, and written once. The clipping takes the chunks in the other order,
// as the last ones that the norm read are still in the last-level cache (310
// million bfloat16: the call 364 against 370 us). Measured there: the norm 136 us
// (4.6 TB/s), the clipping 222 us (5.6 TB/s read and written; a copy reaches 5.2);
// 42 small tensors: 4.3 and 5.2 us of a call of 33 us, which the host's side takes.
#include "device_common.hpp"
#include "internal.hpp"

namespace fp4lin {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 128;
constexpr int64_t kMinChunk = 8192;    // elements
constexpr int64_t kMostChunks = 2048;  // eight workgroups a CU

struct Batch {
  const void* g[kBatch];
  void* out[kBatch];
  int64_t n[kBatch];
  int first[kBatch + 1];  // first chunk of each tensor, within the batch
  uint32_t bf16[kBatch / 32];
  int count;
  int64_t chunk;
};

// Tensor that holds chunk b.
__device__ inline int tensor_of(const Batch& t, int b) {
  int lo = 0, hi = t.count - 1;  // first[lo] <= b < first[hi + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Sum over the workgroup, on every thread, in a fixed order.
__device__ inline double block_sum(double v) {
  __shared__ double sh[kThreads / kWave];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  const int wave = threadIdx.x / kWave;
  if ((threadIdx.x & (kWave - 1)) == 0) sh[wave] = v;
  __syncthreads();
  double s = sh[0];
#pragma unroll
  for (int w = 1; w < kThreads / kWave; ++w) s += sh[w];
  __syncthreads();
  return s;
}

__device__ inline double sum_parts(const double* part, int n) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
  return block_sum(s);
}

template <class In>
__device__ inline double square_sum(const typename In::T* g, int64_t n) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  auto add = [&](const Vec8<In>& v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double x = In::widen(v.v[i]);
      s[i & 3] = fma(x, x, s[i & 3]);
    }
  };
  if ((reinterpret_cast<uintptr_t>(g) & 15) == 0) {
    constexpr int U = 4;  // loads in flight
    const int64_t whole = n / 8;
    int64_t i = threadIdx.x;
    for (; i + (U - 1) * kThreads < whole; i += U * kThreads) {
      Vec8<In> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) load8<In, true>(g + (i + u * kThreads) * 8, 8, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) add(v[u]);
    }
    for (; i < whole; i += kThreads) {
      Vec8<In> v;
      load8<In, true>(g + i * 8, 8, v);
      add(v);
    }
    const int64_t rest = whole * 8 + threadIdx.x;
    if (rest < n) {
      const double x = In::widen(g[rest]);
      s[0] = fma(x, x, s[0]);
    }
  } else {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
      const double x = In::widen(g[i]);
      s[0] = fma(x, x, s[0]);
    }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(Batch t, double* part) {
  const int b = blockIdx.x;
  const int i = tensor_of(t, b);
  const int64_t at = int64_t(b - t.first[i]) * t.chunk;
  const int64_t n = t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk;
  const bool bf16 = (t.bf16[i >> 5] >> (i & 31)) & 1;
  const double s = bf16 ? square_sum<BF16In>(static_cast<const uint16_t*>(t.g[i]) + at, n)
                        : square_sum<F32In>(static_cast<const float*>(t.g[i]) + at, n);
  const double sum = block_sum(s);
  if (threadIdx.x == 0) part[b] = sum;
}

// The sum of n partial sums and its root.
__global__ __launch_bounds__(kThreads) void grad_total_kernel(const double* part, int n,
                                                              double* total, float* norm) {
  const double s = sum_parts(part, n);
  if (threadIdx.x == 0) {
    *total = s;
    *norm = float(sqrt(s));
  }
}

__device__ inline float scaled(float g, float c) { return __fmul_rn(g, c); }
__device__ inline void put(float* p, float v) { *p = v; }
__device__ inline void put(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, __bf16(v));
}

template <class In>
__device__ inline void scale(const typename In::T* g, typename In::T* out, int64_t n, float c) {
  if (((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    constexpr int U = 4;
    const int64_t whole = n / 8;
    auto store = [&](int64_t i, const Vec8<In>& v) {
      __attribute__((aligned(16))) typename In::T o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) put(o + j, scaled(In::widen(v.v[j]), c));
#pragma unroll
      for (int j = 0; j < 8 * In::kBytes; j += 16)
        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(out + i * 8) + j) =
            *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(o) + j);
    };
    int64_t i = threadIdx.x;
    for (; i + (U - 1) * kThreads < whole; i += U * kThreads) {
      Vec8<In> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) load8<In, true>(g + (i + u * kThreads) * 8, 8, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) store(i + u * kThreads, v[u]);
    }
    for (; i < whole; i += kThreads) {
      Vec8<In> v;
      load8<In, true>(g + i * 8, 8, v);
      store(i, v);
    }
    const int64_t rest = whole * 8 + threadIdx.x;
    if (rest < n) put(out + rest, scaled(In::widen(g[rest]), c));
  } else {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) put(out + i, scaled(In::widen(g[i]), c));
  }
}

// part: `parts` partial sums to add here, or (parts = 1) their total. norm: set
// by the first workgroup where it is not NULL.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(Batch t, const double* part,
                                                              int parts, float max_norm,
                                                              float* norm) {
  const float total = float(sqrt(sum_parts(part, parts)));
  const int b = gridDim.x - 1 - blockIdx.x;
  if (norm != nullptr && b == 0 && threadIdx.x == 0) *norm = total;
  float c = max_norm / (total + 1e-6f);
  c = c > 1.0f ? 1.0f : c;  // NaN stays NaN
  const int i = tensor_of(t, b);
  if (c == 1.0f && t.g[i] == t.out[i]) return;
  const int64_t at = int64_t(b - t.first[i]) * t.chunk;
  const int64_t n = t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk;
  if ((t.bf16[i >> 5] >> (i & 31)) & 1)
    scale<BF16In>(static_cast<const uint16_t*>(t.g[i]) + at, static_cast<uint16_t*>(t.out[i]) + at,
                  n, c);
  else
    scale<F32In>(static_cast<const float*>(t.g[i]) + at, static_cast<float*>(t.out[i]) + at, n, c);
}

// The chunks of one batch of tensors (were all batches alike) fit the GPU at once,
// the last, part full chunk of each tensor counted: a few more than fit would run
// alone after the others (310 million bfloat16: the call 370 against 383 us).
int64_t chunk_length(int64_t count, int64_t elements) {
  const int64_t batches = count > 0 ? (count + kBatch - 1) / kBatch : 1;
  const int64_t whole = batches * kMostChunks - count;
  const int64_t c = ((elements + whole - 1) / whole + 63) / 64 * 64;
  return c > kMinChunk ? c : kMinChunk;
}

}  // namespace

int64_t clip_parts(int64_t count, int64_t elements) {
  return elements / chunk_length(count, elements) + count;
}

hipError_t launch_clip(const fp4lin_grad* grads, int64_t count, int64_t elements, bool clip,
                       float max_norm, float* norm, void* ws, hipStream_t stream) {
  double* const total = static_cast<double*>(ws);
  double* const part = total + 2;  // 16 bytes on
  const int64_t chunk = chunk_length(count, elements);
  auto fill = [&](Batch& t, int64_t& next) {
    t = Batch{};
    t.chunk = chunk;
    for (; next < count && t.count < kBatch; ++next) {
      const fp4lin_grad& x = grads[next];
      if (x.n == 0) continue;
      const int i = t.count++;
      t.g[i] = x.g;
      t.out[i] = x.out;
      t.n[i] = x.n;
      if (x.dt == FP4LIN_BF16) t.bf16[i >> 5] |= 1u << (i & 31);
      t.first[i + 1] = t.first[i] + int((x.n + chunk - 1) / chunk);
    }
  };
  Batch t;
  int64_t next = 0, parts = 0, batches = 0;
  do {
    fill(t, next);
    if (t.count == 0) break;
    const int blocks = t.first[t.count];
    grad_norm_kernel<<<unsigned(blocks), kThreads, 0, stream>>>(t, part + parts);
    parts += blocks;
    ++batches;
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } while (next < count);
  const bool inside = clip && batches == 1;  // the clipping kernel adds the sums
  if (!inside) {
    grad_total_kernel<<<1, kThreads, 0, stream>>>(part, int(parts), total, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!clip) return hipSuccess;
  next = 0;
  for (int64_t k = 0; k < batches; ++k) {
    fill(t, next);
    grad_scale_kernel<<<unsigned(t.first[t.count]), kThreads, 0, stream>>>(
        t, inside ? part : total, inside ? int(parts) : 1, max_norm, inside ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4lin
