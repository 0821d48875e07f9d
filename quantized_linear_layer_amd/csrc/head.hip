// Softmax cross entropy of a large vocabulary straight from the hidden states,
// with its gradients: the T x V logits are never in memory as a whole.
//
//   l = X W                     X: T x H, W: H x V (or stored V x H)
//   lse_t  = log sum_v exp l_tv
//   loss_t = lse_t - l_(t, target_t)          0 for a target outside [0, V)
//   G_tv   = (exp(l_tv - lse_t) - [v = target_t]) * dloss_t     likewise 0
//   dX = G W^T,  dW = X^T G
//
// Forward: one product whose tiles keep, of each row, the maximum and the sum of
// exponentials over the columns of a wave (fp32), and the target's logit where
// the tile holds it; a second kernel joins the columns' pairs (m, s) of a row as
//   M = max m_i,  lse = M + log sum_i s_i exp(m_i - M).
//
// Backward, in pieces of the vocabulary: the piece's logits are formed again,
// turned into G in the tile's epilogue and written in the inputs' type, then
// multiplied into dX (fp32, added up over the pieces) and into the piece's own
// part of dW. A piece is as wide as lets its G stay in the last-level cache
// between the three products (kPieceBytes), which is also what bounds the
// workspace. G is rounded once to the inputs' type (bfloat16: 2^-9 of each
// element, as the two products it feeds take bfloat16 operands); every sum is
// fp32. Both sides of that choice, bfloat16 4096 x 2048 and 8192 x 4096 by 32000: as it
// is the gradients are off by 0.0019 of their norm, and loss and gradients take 1.93
// and 7.16 ms; with G in two bfloat16 parts, which makes both products twice as long,
// they are off by 0.0017, their own rounding to bfloat16 alone, and take 2.88 and 10.73.
//
// dX sums over the vocabulary, so few rows leave few tiles: the reduction is
// then split over workgroups, each adding into an fp32 array of its own, and the
// arrays are added in a fixed order at the end. No atomics: results repeat bit
// for bit.
//
// Operands whose rows do not start on 16 bytes or whose contiguous size is not a
// multiple of 8 elements are first copied, padded with zeros. The backward always
// takes a copy of X, in which the rows that are left out are zero: what they hold,
// infinities and NaN included, reaches no gradient.
#include <type_traits>

#include "dense_core.hpp"
#include "device_common.hpp"
#include "gemm_core.hpp"
#include "internal.hpp"

namespace fp4lin {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ inline float exp_diff(float x, float y) {
  return __builtin_amdgcn_exp2f((x - y) * kLog2e);
}

// Reductions over the 32 lanes of a half wave, on every lane and on the vector
// unit: four exchanges within rows of 16 lanes (neighbours, pairs, mirrored 8,
// mirrored 16), then the two rows of a half (v_permlane16_swap).
template <class Op>
__device__ inline float half_reduce(float v, const Op& op) {
  auto dpp = [](float x, auto ctrl) {
    const int i = __float_as_int(x);
    return __int_as_float(__builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = op(v, dpp(v, std::integral_constant<int, 0xb1>{}));   // quad_perm [1, 0, 3, 2]
  v = op(v, dpp(v, std::integral_constant<int, 0x4e>{}));   // quad_perm [2, 3, 0, 1]
  v = op(v, dpp(v, std::integral_constant<int, 0x141>{}));  // row_half_mirror
  v = op(v, dpp(v, std::integral_constant<int, 0x140>{}));  // row_mirror
  const auto sw = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(sw[0]), __uint_as_float(sw[1]));
}
__device__ inline float half_max(float v) {
  return half_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float half_sum(float v) {
  return half_reduce(v, [](float a, float b) { return a + b; });
}

// Row of element r of a 32x32 fragment on this lane.
__device__ inline int frag_row(int r, int lane) { return 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3); }

// LDS stages of a tile: eight waves have a CU to themselves and take turns on
// all of its LDS; tiles of few rows keep more steps on their way, those of 64 x 64
// as many as let five of them have a CU together.
template <class C>
constexpr int kStages = C::kThreads == 512 ? 5 : C::BM == 64 ? (C::BN == 64 ? 4 : 5) : 3;

template <class C, class F>
__device__ __attribute__((always_inline)) inline void product_tile(F& f, int nkt, uint8_t* st0,
                                                                   uint8_t* st1, uint8_t* st2,
                                                                   uint8_t* st3, uint8_t* st4) {
  uint8_t* const st[5] = {st0, st1, st2, st3, st4};
  if constexpr (C::kThreads == 512)
    gemm_pipeline_turns<F, 5>(f, nkt, st);
  else if constexpr (kStages<C> == 5)
    gemm_pipeline_deep<F, 5>(f, nkt, st);
  else if constexpr (kStages<C> == 4)
    gemm_pipeline_deep<F, 4>(f, nkt, {st0, st1, st2, st3});
  else
    gemm_pipeline(f, nkt, st0, st1, st2);
}

template <class T>
struct HeadArgs {
  DenseOperand<T> X, W;  // W: extent V
  int T_, V, H;          // rows, columns, reduction
  int v0, Vall;          // W's first column in the vocabulary, and its size
  const int32_t* target;
  // forward
  float2* part;     // [T][parts]: (m, s) of each group of columns
  int parts;
  float* tlogit;    // [T]
  // backward
  const float* lse;
  const float* dloss;
  const float* top;  // G's scale, see head_prepare_kernel
  T* G;
  int64_t ldg;
};

// One (m, s) a row and wave, and the targets' logits. Bound by the matrix core and
// its clock under load: 8192 x 4096 by 32000 in bfloat16 1.83 ms (1.18 PFLOP/s, the
// matrix core busy 0.77 at 1.63 GHz; a library's plain product of the size reaches
// 1.42). The pair leaves instead of 256 columns of logits, so the tile's way out is
// 8 bytes a row and wave. With 32 rows the kernel is a read of W: 43 us for 262 MB
// (6.1 TB/s). float32 1001 x 515 by 5003: 64 us (81 TFLOP/s).
template <class C, class T, int kBT>
__global__ __launch_bounds__(C::kThreads, C::kMinBlocks) void head_lse_kernel(HeadArgs<T> p) {
  constexpr int FM = C::FM, FN = C::FN;
  __shared__ __attribute__((aligned(16))) uint8_t st0[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st1[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st2[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st3[kStages<C> > 3 ? C::kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t st4[kStages<C> > 4 ? C::kStageBytes : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int tiles_m = (p.T_ + C::BM - 1) / C::BM, tiles_n = (p.V + C::BN - 1) / C::BN;
  int tm, tn;
  tile_of(xcd_run(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  DenseFeed<C, T, kAlong, kBT> f(p.X, p.W, m0, n0, wave, lane);
  product_tile<C>(f, (p.H + kStepElems<T> - 1) / kStepElems<T>, st0, st1, st2, st3, st4);

  const int row0 = m0 + wm * FM * 32, col0 = n0 + wn * FN * 32;
  // the rows of this wave whose target it holds: few, so they are looked up one
  // by one among the accumulators
  const int trow = row0 + lane;
  const int tcol = lane < FM * 32 && trow < p.T_ ? p.target[trow] : -1;
  uint64_t hits = __ballot(tcol >= col0 && tcol < col0 + FN * 32 && tcol < p.V);
  while (hits != 0) {
    const int l = __builtin_ctzll(hits);
    hits &= hits - 1;
    const int c = __builtin_amdgcn_readlane(tcol, l) - col0;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (fm * 32 + frag_row(r, lane) == l && fn * 32 + (lane & 31) == c)
            p.tlogit[row0 + l] = f.acc[fm][fn][r];
  }
  // columns past the vocabulary count as -inf
#pragma unroll
  for (int fn = 0; fn < FN; ++fn)
    if (col0 + fn * 32 + (lane & 31) >= p.V) {
#pragma unroll
      for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int r = 0; r < 16; ++r) f.acc[fm][fn][r] = -__builtin_huge_valf();
    }
  float2* const part = p.part + (tn * C::WN + wn);
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float m = f.acc[fm][0][r];
#pragma unroll
      for (int fn = 1; fn < FN; ++fn) m = fmaxf(m, f.acc[fm][fn][r]);
      m = half_max(m);
      const float ref = m == -__builtin_huge_valf() ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) s += exp_diff(f.acc[fm][fn][r], ref);
      s = half_sum(s);
      const int row = row0 + fm * 32 + frag_row(r, lane);
      if ((lane & 31) == 0 && row < p.T_) part[int64_t(row) * p.parts] = make_float2(m, s);
    }
}

// Joins a row's P pairs: one wave a row, so that few rows with many pairs (32 rows,
// 1000 pairs: 7.6 us; one thread a row: 75) wait for few loads in a row.
constexpr int kJoinRows = 4;

__global__ __launch_bounds__(kJoinRows * 64) void head_join_kernel(
    const float2* __restrict__ part, int P, int T, int V, const int32_t* __restrict__ target,
    const float* __restrict__ tlogit, float* __restrict__ loss, float* __restrict__ lse) {
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.x * kJoinRows + (threadIdx.x >> 6);
  if (row >= T) return;
  float m = -__builtin_huge_valf(), s = 0.0f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float ref = top == -__builtin_huge_valf() ? 0.0f : top;
    s = s * exp_diff(m, ref) + s2 * exp_diff(m2, ref);
    m = top;
  };
  const float2* const mine = part + int64_t(row) * P;
  for (int j = lane; j < P; j += 64) join(mine[j].x, mine[j].y);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float m2 = __shfl_xor(m, off, kWave), s2 = __shfl_xor(s, off, kWave);
    join(m2, s2);
  }
  if (lane != 0) return;
  const float l = m + logf(s);
  lse[row] = l;
  const int t = target[row];
  loss[row] = t >= 0 && t < V ? l - tlogit[row] : 0.0f;
}

// bfloat16 G is kept in pieces of 32 columns, the rows of a piece together: the
// order in which dX reads it along (kAlong, a K step's rows together) and dW
// across (kPieces) in whole cache lines. float32 G is kept by rows.
template <class T>
constexpr bool kGPieces = sizeof(T) == 2;

// G of a piece of the vocabulary over the largest |dloss|, zeros in the columns
// that pad it to a multiple of 32 (float32: 8). As head_lse_kernel bound by the
// matrix core: 8192 x 4096 by 8192 columns in 471 us (1.17 PFLOP/s).
template <class C, class T, int kBT>
__global__ __launch_bounds__(C::kThreads, C::kMinBlocks) void head_grad_kernel(HeadArgs<T> p) {
  constexpr int FM = C::FM, FN = C::FN;
  __shared__ __attribute__((aligned(16))) uint8_t st0[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st1[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st2[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st3[kStages<C> > 3 ? C::kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t st4[kStages<C> > 4 ? C::kStageBytes : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int tiles_m = (p.T_ + C::BM - 1) / C::BM, tiles_n = (p.V + C::BN - 1) / C::BN;
  int tm, tn;
  tile_of(xcd_run(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  DenseFeed<C, T, kAlong, kBT> f(p.X, p.W, m0, n0, wave, lane);
  product_tile<C>(f, (p.H + kStepElems<T> - 1) / kStepElems<T>, st0, st1, st2, st3, st4);

  const int row0 = m0 + wm * FM * 32, col0 = n0 + wn * FN * 32;
  float g[FM][16];  // dloss of this lane's rows over the largest
  const float top = *p.top;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = row0 + fm * 32 + frag_row(r, lane);
      const int at = row < p.T_ ? row : p.T_ - 1;
      const float lse = p.lse[at];
      const int t = p.target[at];
      g[fm][r] = p.dloss[at] / top;
      // a row that is left out: zeros, whatever its lse and dloss
      const bool out = t < 0 || t >= p.Vall;
      if (out) g[fm][r] = 0.0f;
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        f.acc[fm][fn][r] = out ? 0.0f : exp_diff(f.acc[fm][fn][r], lse);
    }
  // the one-hot part, as in head_lse_kernel
  const int trow = row0 + lane;
  const int tcol = lane < FM * 32 && trow < p.T_ ? p.target[trow] : -1;
  uint64_t hits = __ballot(tcol >= p.v0 + col0 && tcol < p.v0 + col0 + FN * 32);
  while (hits != 0) {
    const int l = __builtin_ctzll(hits);
    hits &= hits - 1;
    const int c = __builtin_amdgcn_readlane(tcol, l) - p.v0 - col0;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (fm * 32 + frag_row(r, lane) == l && fn * 32 + (lane & 31) == c)
            f.acc[fm][fn][r] -= 1.0f;
  }
  // columns past the piece: the zeros that pad G
#pragma unroll
  for (int fn = 0; fn < FN; ++fn)
    if (col0 + fn * 32 + (lane & 31) >= p.V) {
#pragma unroll
      for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int r = 0; r < 16; ++r) f.acc[fm][fn][r] = 0.0f;
    }
  const int cols = kGPieces<T> ? (p.V + 31) & ~31 : (p.V + 7) & ~7;
  emit_tile<C, kOutVec<T>>(
      st0, st1, st2, wave, lane, m0, n0,
      [&](int fm, int fn, int r) { return f.acc[fm][fn][r] * g[fm][r]; },
      [&](int gr, int gc, const float* v) {
        if (gr >= p.T_) return;
        T* const dst = kGPieces<T> ? p.G + (gc / 32 * int64_t(p.T_) + gr) * 32 + gc % 32
                                   : p.G + int64_t(gr) * p.ldg + gc;
        store_vec<false>(dst, v, cols - gc, true);
      });
}

// Elements from an operand's reduction element 0 to k0, a multiple of a K step.
template <class C, class T, int kT>
__device__ inline int64_t at_step(const DenseOperand<T>& o, int k0) {
  return kT == kAlong ? k0 / kStepElems<T> * o.step : kT == kAcross ? k0 * o.ld : int64_t(k0) * 32;
}

// A product of two operands, or of slice blockIdx.z of their reduction. kAdd: into
// the fp32 array of the slice (Y + z * slice_elems), on top of what is there
// unless `first`. Measured on a piece of 8192 columns, 8192 x 4096 in bfloat16: dX
// 461 us (1.19 PFLOP/s, matrix core busy 0.76), dW 427 us (1.29, busy 0.82; both
// operands are read in whole cache lines).
template <class T, class Out>
struct ProductArgs {
  DenseOperand<T> A, B;
  int M, N;     // output
  int k_slice;  // reduction elements a slice (whole K steps)
  Out* Y;
  int64_t ldy;
  int64_t slice_elems;
  int first;
  const float* scale;  // of the result (not of the slices' arrays)
};

template <class C, class T, int kAT, int kBT, class Out, bool kAdd>
__global__ __launch_bounds__(C::kThreads, C::kMinBlocks) void head_product_kernel(
    ProductArgs<T, Out> p) {
  __shared__ __attribute__((aligned(16))) uint8_t st0[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st1[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st2[C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t st3[kStages<C> > 3 ? C::kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t st4[kStages<C> > 4 ? C::kStageBytes : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_m = (p.M + C::BM - 1) / C::BM, tiles_n = (p.N + C::BN - 1) / C::BN;
  int tm, tn;
  tile_of(xcd_run(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int k0 = blockIdx.z * p.k_slice;
  DenseOperand<T> A = p.A, B = p.B;
  A.p += at_step<C, T, kAT>(A, k0);
  B.p += at_step<C, T, kBT>(B, k0);
  A.k = A.k - k0 < p.k_slice ? A.k - k0 : p.k_slice;
  B.k = B.k - k0 < p.k_slice ? B.k - k0 : p.k_slice;
  // (one of the two may be filled up to a multiple of 8 with zeros; the other
  // then reads as zero there)
  const int k = A.k > B.k ? A.k : B.k;
  DenseFeed<C, T, kAT, kBT> f(A, B, m0, n0, wave, lane);
  constexpr int kE = kStepElems<T>;
  if (k > 0) product_tile<C>(f, (k + kE - 1) / kE, st0, st1, st2, st3, st4);
  Out* const Y = p.Y + blockIdx.z * p.slice_elems;
  const bool vec = rows_vec(Y, p.ldy);
  float scale = 1.0f;
  if constexpr (!kAdd) scale = *p.scale;
  emit_tile<C, kOutVec<Out>>(
      st0, st1, st2, wave, lane, m0, n0,
      [&](int fm, int fn, int r) { return kAdd ? f.acc[fm][fn][r] : f.acc[fm][fn][r] * scale; },
      [&](int gr, int gc, const float* v) {
        if (gr >= p.M) return;
        Out* const dst = Y + int64_t(gr) * p.ldy + gc;
        if constexpr (kAdd) {
          // H is padded to whole 16-byte groups in this array
          if (gc >= p.ldy) return;
          f32x4 o = {v[0], v[1], v[2], v[3]};
          if (!p.first) o += *reinterpret_cast<const f32x4*>(dst);
          *reinterpret_cast<f32x4*>(dst) = o;
        } else {
          store_vec<true>(dst, v, p.N - gc, vec);
        }
      });
}

// dX from the S arrays of its slices (T x ldp each), added in slice order, times
// *scale. Bound by memory: 33.7 us for 8192 x 4096 from one array (6 TB/s).
template <class Out>
__global__ __launch_bounds__(256) void head_sum_kernel(const float* __restrict__ acc, int S,
                                                       int64_t slice_elems, int64_t T, int H,
                                                       int64_t ldp, const float* __restrict__ scale,
                                                       Out* __restrict__ dX, int64_t lddx) {
  const float g = *scale;
  const int64_t groups = ldp / 4;
  const bool vec = (reinterpret_cast<uintptr_t>(dX) % (4 * sizeof(Out)) == 0) && lddx % 4 == 0;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < T * groups;
       i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / groups;
    const int c = int(i - row * groups) * 4;
    f32x4 o = *reinterpret_cast<const f32x4*>(acc + row * ldp + c);
    for (int s = 1; s < S; ++s)
      o += *reinterpret_cast<const f32x4*>(acc + s * slice_elems + row * ldp + c);
    o *= g;
    Out* const dst = dX + row * lddx + c;
    if constexpr (sizeof(Out) == 4) {
      if (vec && c + 4 <= H) {
        *reinterpret_cast<f32x4*>(dst) = o;
        continue;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < H) dst[j] = o[j];
    } else {
      const uint32_t u[2] = {bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
      if (vec && c + 4 <= H) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
        continue;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < H) dst[j] = uint16_t(u[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// What the products need first, in one launch: copies of X and W where they have
// to be, and for the backward the largest finite |dloss| of the rows whose target
// lies in the vocabulary, 1 if that is 0 (the last workgroup). An infinite dloss is
// left to its own row: as the scale it would make NaN of the others' zeros. Why a
// scale: a mean's dloss is one number in all rows, and rounded into bfloat16 G it
// would be off alike everywhere (0.0032 of the gradients' norm at 4096 x 2048 by
// 32000; 0.0019 with G over it). 27 us for 8192 x 4096 (67 MB read and written).
template <class T>
struct PackArgs {
  const T* src;
  int64_t R, C, ld;
  T* dst;
  int64_t ldp;   // a multiple of 8 (steps: of 32); zeros from the C-th element on
  int steps;     // the rows of 32 columns together (kAlong's second form), not rows of ldp
  int blocks;    // 0: no copy
  const int32_t* target;  // not NULL: zeros in the rows whose target is not in [0, V)
  int V;

  __device__ int64_t columns(int64_t row) const {
    if (target == nullptr) return C;
    const int t = target[row];
    return t >= 0 && t < V ? C : 0;
  }
};

template <class T>
struct PrepareArgs {
  PackArgs<T> x, w;
  const float* dloss;
  const int32_t* target;
  int T_, V;
  float* top;
};

// One thread per 8 elements of the copy.
template <class T>
__device__ inline void pack(const PackArgs<T>& p, int block) {
  const int64_t groups = p.ldp / 8;
  for (int64_t i = int64_t(block) * 256 + threadIdx.x; i < p.R * groups;
       i += int64_t(p.blocks) * 256) {
    const int64_t row = i / groups, c = (i - row * groups) * 8, C = p.columns(row);
    __attribute__((aligned(16))) T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < C ? p.src[row * p.ld + c + j] : T(0);
    T* const dst = p.dst + row * p.ldp + c;
#pragma unroll
    for (int j = 0; j < 8 * int(sizeof(T)); j += 16)
      *reinterpret_cast<uint4*>(reinterpret_cast<char*>(dst) + j) =
          *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(v) + j);
  }
}

// The same with the rows of 32 columns together (bfloat16): a wave takes 16 rows,
// four lanes each, and four steps of them at a time, so that it reads 256 bytes of
// a row and writes 1 KiB in one piece.
__device__ inline void pack_steps(const PackArgs<uint16_t>& p, int block) {
  const int lane = threadIdx.x & 63;
  const int64_t quads = (p.ldp / 32 + 3) / 4, tiles = (p.R + 15) / 16 * quads;
  const bool fast = reinterpret_cast<uintptr_t>(p.src) % 16 == 0 && p.ld % 8 == 0 && p.C % 8 == 0;
  for (int64_t t = int64_t(block) * 4 + (threadIdx.x >> 6); t < tiles; t += int64_t(p.blocks) * 4) {
    const int64_t r0 = t / quads * 16, s0 = (t - t / quads * quads) * 4;
    const int64_t row = r0 + (lane >> 2);
    if (row >= p.R) continue;
    const int64_t C = p.columns(row);
    Vec8<BF16In> v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t c = (s0 + u) * 32 + (lane & 3) * 8;
      if (fast)
        load_chunk<BF16In, true>(p.src + row * p.ld, c < C ? c : p.C, p.C, v[u]);
      else
        load_chunk<BF16In, false>(p.src + row * p.ld, c, C, v[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if ((s0 + u) * 32 >= p.ldp) break;
      uint4 o;
      o.x = v[u].v[0] | uint32_t(v[u].v[1]) << 16;
      o.y = v[u].v[2] | uint32_t(v[u].v[3]) << 16;
      o.z = v[u].v[4] | uint32_t(v[u].v[5]) << 16;
      o.w = v[u].v[6] | uint32_t(v[u].v[7]) << 16;
      *reinterpret_cast<uint4*>(p.dst + ((s0 + u) * p.R + row) * 32 + (lane & 3) * 8) = o;
    }
  }
}

template <class T>
__global__ __launch_bounds__(256) void head_prepare_kernel(PrepareArgs<T> p) {
  const int b = blockIdx.x;
  if (b < p.x.blocks) {
    if constexpr (sizeof(T) == 2)
      if (p.x.steps) return pack_steps(p.x, b);
    return pack(p.x, b);
  }
  if (b < p.x.blocks + p.w.blocks) return pack(p.w, b - p.x.blocks);
  __shared__ float sh[4];
  float m = 0.0f;
  constexpr int U = 8;  // rows in flight a thread
  for (int i0 = threadIdx.x; i0 < p.T_; i0 += 256 * U) {
    float g[U];
    int t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256 < p.T_ ? i0 + u * 256 : p.T_ - 1;
      g[u] = p.dloss[i];
      t[u] = p.target[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t[u] >= 0 && t[u] < p.V && fabsf(g[u]) < __builtin_huge_valf()) m = fmaxf(m, fabsf(g[u]));
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    m = fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
    *p.top = m != 0.0f ? m : 1.0f;
  }
}

// ---------------------------------------------------------------------------
// Host: tiles, pieces, slices.
// ---------------------------------------------------------------------------
using LargeTile = GemmCfg<256, 256, 4, 2, 64, 1>;
using MidTile = GemmCfg<128, 256, 2, 2, 64, 2>;
using FewTile = GemmCfg<64, 128, 1, 4, 64, 2>;
using F32Tile = GemmCfg<128, 128, 2, 2, 64, 2>;
using F32Small = GemmCfg<64, 64, 2, 2, 64, 4>;

// Bytes of G. Loss and gradients by 32000 columns of 4096 x 2048 and 8192 x 4096:
// 64 MB 1940 and 7243 us, 128 MB 1851 and 6912, 256 MB 1840 and 6934.
constexpr int64_t kPieceBytes = int64_t(128) << 20;
constexpr int64_t kCUs = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t round32(int64_t n) { return (n + 31) / 32 * 32; }
int64_t round_256(int64_t n) { return (n + 255) / 256 * 256; }

unsigned copy_blocks(int64_t threads) {
  const int64_t b = ceil_div(threads, 256);
  return unsigned(b < 4096 ? (b > 0 ? b : 1) : 4096);
}

enum class Tile { kLarge, kMid, kFew, kF32, kF32Small };

int64_t tile_rows(Tile t) {
  return t == Tile::kLarge ? 256 : t == Tile::kMid || t == Tile::kF32 ? 128 : 64;
}
int64_t tile_cols(Tile t) {
  return t == Tile::kLarge || t == Tile::kMid ? 256 : t == Tile::kF32Small ? 64 : 128;
}
// columns of a wave
int64_t wave_cols(Tile t) {
  return t == Tile::kLarge || t == Tile::kMid ? 128 : t == Tile::kF32 ? 64 : 32;
}
int64_t tiles_of(Tile t, int64_t M, int64_t N) {
  return ceil_div(M, tile_rows(t)) * ceil_div(N, tile_cols(t));
}

// Tile of an M x N product and the slices its reduction is cut in (at most `most`).
struct Shape {
  Tile tile;
  int64_t slices;
};

// bfloat16: 256 x 256 once those give every CU one, and as many slices as give
// every CU a workgroup (of 256 x 256) or two; else 128 x 256. Loss and gradients,
// 256 x 256 wherever possible / 128 x 256 / the rule: 512x1024x16000 145 / 135 / 135
// us, 256x2048x32000 235 / 218 / 218, 1024x2048x32000 521 / 556 / 521; the loss alone
// of 2048x4096x32000 459 / 525 / 459. 64 x 128 for up to 64 rows: up to 256 of them
// 263 us for 256x2048x32000.
// float32, whose products are bound by the matrix core: the tile and the slices
// whose busiest CU has least to do, of equal ones the larger tile and the fewer
// slices, which read and add less; two workgroups a CU where slices can give them.
// Measured, loss and gradients of T x H x V, all three tiles against the larger
// two: 1001x515x5003 237 against 294 us, 300x256x3000 57 against 87,
// 700x1000x10000 494 against 541.
Shape pick(bool bf16, int64_t M, int64_t N, int64_t most) {
  if (bf16 || M <= 64) {
    const Tile t = M <= 64 ? Tile::kFew
                   : M > 128 && tiles_of(Tile::kLarge, M, N) * most >= kCUs ? Tile::kLarge
                                                                            : Tile::kMid;
    const int64_t want = ceil_div((t == Tile::kLarge ? 1 : 2) * kCUs, tiles_of(t, M > 0 ? M : 1, N));
    return Shape{t, want < most ? want : most};
  }
  Shape best{};
  double least = 0.0;
  for (Tile t : {Tile::kF32, Tile::kFew, Tile::kF32Small}) {
    const int64_t tiles = tiles_of(t, M, N);
    for (int64_t s = 1; s <= most && (s == 1 || tiles * s <= 4 * kCUs); ++s) {
      if (s < most && tiles * s < 2 * kCUs) continue;
      const double work = double(ceil_div(tiles * s, kCUs) * tile_rows(t) * tile_cols(t)) / double(s);
      if (least == 0.0 || work < least) {
        least = work;
        best = Shape{t, s};
      }
    }
  }
  return best;
}
Tile pick_tile(bool bf16, int64_t M, int64_t N) { return pick(bf16, M, N, 1).tile; }

// dX (T x H, reduction over the k columns of a piece): slices of at least 512, so
// that a slice's sum is longer than its way out.
constexpr int64_t kSliceElems = 512, kMaxSlices = 32;

Shape pick_dx(bool bf16, int64_t T, int64_t H, int64_t k) {
  const int64_t most = k / kSliceElems > 1 ? k / kSliceElems : 1;
  return pick(bf16, T, H, most < kMaxSlices ? most : kMaxSlices);
}

// f(tile configuration) for a tile that pick_tile gives for T.
template <class T, class F>
hipError_t with_tile(Tile t, F&& f) {
  if (t == Tile::kFew) return f(FewTile{});
  if constexpr (sizeof(T) == 2) {
    if (t == Tile::kLarge) return f(LargeTile{});
    if (t == Tile::kMid) return f(MidTile{});
  } else {
    if (t == Tile::kF32) return f(F32Tile{});
    if (t == Tile::kF32Small) return f(F32Small{});
  }
  return hipErrorInvalidValue;
}

}  // namespace

HeadPlan head_plan(bool bf16, bool backward, int64_t T, int64_t H, int64_t V, bool by_vocab,
                   int64_t ldx, int64_t ldw) {
  const int64_t esz = bf16 ? 2 : 4;
  HeadPlan h{};
  h.pack_x = backward || H % 8 != 0 || (ldx * esz) % 16 != 0;
  h.pack_w = (by_vocab ? H : V) % 8 != 0 || (ldw * esz) % 16 != 0;
  // bfloat16: X with a K step's rows together, for the logits of more than a few
  // rows and as dW's operand (copied / not: the loss of 256x4096x32000 98 / 103 us,
  // of 2048x4096x32000 459 / 484, of 64x4096x32000 66 / 62)
  h.step_x = bf16 && (backward || T > 64);
  h.pack_x = h.pack_x && !h.step_x;
  h.ldx = h.pack_x ? round8(H) : ldx;
  h.ldw = h.pack_w ? round8(by_vocab ? H : V) : ldw;
  h.x_bytes = h.step_x ? T * round32(H) * esz : h.pack_x ? T * h.ldx * esz : 0;
  h.w_bytes = h.pack_w ? (by_vocab ? V : H) * h.ldw * esz : 0;
  const Tile t = pick_tile(bf16, T, V);
  h.parts = ceil_div(V, tile_cols(t)) * (tile_cols(t) / wave_cols(t));
  const int64_t pieces = ceil_div(T * V * esz, kPieceBytes);
  h.piece = pieces > 1 ? round_256(ceil_div(V, pieces)) : V;
  h.ldg = bf16 ? round32(h.piece) : round8(h.piece);
  h.slices = pick_dx(bf16, T, H, h.piece).slices;
  h.ldp = round8(H);
  return h;
}

namespace {

// X and W as the products take them, copied where they have to be; for the
// backward the largest |dloss| besides. X: as the logits read it.
template <class T>
hipError_t prepare(const HeadCall& c, const HeadPlan& h, bool backward, DenseOperand<T>* X,
                   const T** W, hipStream_t stream) {
  const T* const x = static_cast<const T*>(c.X);
  const T* const w = static_cast<const T*>(c.W);
  T* const xc = static_cast<T*>(c.packed_x);
  const int64_t wr = c.by_vocab ? c.V : c.H, wc = c.by_vocab ? c.H : c.V;
  PrepareArgs<T> p{};
  if (h.step_x && c.T > 0)
    p.x = PackArgs<T>{x, c.T, c.H, c.ldx, xc, round32(c.H), 1,
                      int(copy_blocks(ceil_div(c.T, 16) * ceil_div(c.H, 128) * 64)), nullptr, 0};
  else if (h.pack_x && c.T > 0)
    p.x = PackArgs<T>{x, c.T, c.H, c.ldx, xc, h.ldx, 0, int(copy_blocks(c.T * (h.ldx / 8))),
                      nullptr, 0};
  if (backward) {
    p.x.target = c.target;
    p.x.V = int(c.V);
  }
  if (h.pack_w)
    p.w = PackArgs<T>{w, wr, wc, c.ldw, static_cast<T*>(c.packed_w), h.ldw, 0,
                      int(copy_blocks(wr * (h.ldw / 8))), nullptr, 0};
  p.dloss = c.dloss;
  p.target = c.target;
  p.T_ = int(c.T);
  p.V = int(c.V);
  p.top = c.top;
  const int blocks = p.x.blocks + p.w.blocks + (backward ? 1 : 0);
  if (blocks > 0) head_prepare_kernel<T><<<unsigned(blocks), 256, 0, stream>>>(p);
  constexpr int kE = kStepElems<T>;
  *X = h.step_x ? DenseOperand<T>{xc, kE, c.T * kE, int(c.T), int(round32(c.H))}
                : DenseOperand<T>{h.pack_x ? xc : x, h.ldx, kE, int(c.T), int(round8(c.H))};
  *W = h.pack_w ? static_cast<const T*>(c.packed_w) : w;
  return hipGetLastError();
}

// Columns v0 .. v0 + n - 1 of the vocabulary as the logits read W's.
template <class T>
DenseOperand<T> weight_columns(const HeadCall& c, const HeadPlan& h, const T* W, int64_t v0,
                               int64_t n) {
  if (c.by_vocab)
    return DenseOperand<T>{W + v0 * h.ldw, h.ldw, kStepElems<T>, int(n), int(round8(c.H))};
  return DenseOperand<T>{W + v0, h.ldw, 0, int(round8(n)), int(c.H)};
}

template <class T, bool kGrad>
hipError_t logits(Tile t, bool by_vocab, const HeadArgs<T>& a, hipStream_t stream) {
  const int64_t tiles = tiles_of(t, a.T_, a.V);
  if (tiles >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  return with_tile<T>(t, [&](auto c) -> hipError_t {
    using C = decltype(c);
    const dim3 grid(unsigned(tiles), 1, 1);
    if constexpr (kGrad) {
      if (by_vocab)
        head_grad_kernel<C, T, kAlong><<<grid, C::kThreads, 0, stream>>>(a);
      else
        head_grad_kernel<C, T, kAcross><<<grid, C::kThreads, 0, stream>>>(a);
    } else {
      if (by_vocab)
        head_lse_kernel<C, T, kAlong><<<grid, C::kThreads, 0, stream>>>(a);
      else
        head_lse_kernel<C, T, kAcross><<<grid, C::kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
  });
}

template <class T, int kAT, int kBT, class Out, bool kAdd>
hipError_t product(Tile t, const ProductArgs<T, Out>& a, int64_t slices, hipStream_t stream) {
  return with_tile<T>(t, [&](auto c) -> hipError_t {
    using C = decltype(c);
    const dim3 grid(unsigned(tiles_of(t, a.M, a.N)), 1, unsigned(slices));
    head_product_kernel<C, T, kAT, kBT, Out, kAdd><<<grid, C::kThreads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

template <class T>
hipError_t run_forward(const HeadCall& c, const HeadPlan& h, hipStream_t stream) {
  DenseOperand<T> X;
  const T* W;
  hipError_t e = prepare<T>(c, h, false, &X, &W, stream);
  if (e != hipSuccess) return e;
  HeadArgs<T> a{};
  a.X = X;
  a.W = weight_columns(c, h, W, 0, c.V);
  a.T_ = int(c.T);
  a.V = a.Vall = int(c.V);
  a.H = int(c.H);
  a.target = c.target;
  a.part = static_cast<float2*>(c.part);
  a.parts = int(h.parts);
  a.tlogit = c.tlogit;
  e = logits<T, false>(pick_tile(sizeof(T) == 2, c.T, c.V), c.by_vocab, a, stream);
  if (e != hipSuccess) return e;
  head_join_kernel<<<unsigned(ceil_div(c.T, kJoinRows)), kJoinRows * 64, 0, stream>>>(
      a.part, int(h.parts), int(c.T), int(c.V), c.target, c.tlogit, c.loss, c.lse_out);
  return hipGetLastError();
}

template <class T>
hipError_t run_backward(const HeadCall& c, const HeadPlan& h, hipStream_t stream) {
  constexpr bool kBf16 = sizeof(T) == 2;
  DenseOperand<T> X;
  const T* W;
  hipError_t e = prepare<T>(c, h, true, &X, &W, stream);
  if (e != hipSuccess) return e;
  T* const dW = static_cast<T*>(c.dW);
  const Tile tx = pick_dx(kBf16, c.T, c.H, h.piece).tile;
  const bool direct = h.slices == 1 && h.piece >= c.V;
  for (int64_t v0 = 0; v0 < c.V; v0 += h.piece) {
    const int64_t n = c.V - v0 < h.piece ? c.V - v0 : h.piece;
    const int n8 = int(round8(n));
    T* const G = static_cast<T*>(c.G);
    if (c.T > 0) {
      HeadArgs<T> a{};
      a.X = X;
      a.W = weight_columns(c, h, W, v0, n);
      a.T_ = int(c.T);
      a.V = int(n);
      a.Vall = int(c.V);
      a.H = int(c.H);
      a.v0 = int(v0);
      a.target = c.target;
      a.lse = c.lse;
      a.dloss = c.dloss;
      a.top = c.top;
      a.G = G;
      a.ldg = h.ldg;
      e = logits<T, true>(pick_tile(kBf16, c.T, n), c.by_vocab, a, stream);
      if (e != hipSuccess) return e;

      // dX: G (T x n) times W's piece transposed; the columns that fill n to n8 are
      // zeros in G and, where W is read along them, in W
      constexpr int kE = kStepElems<T>;
      const DenseOperand<T> A = kGPieces<T> ? DenseOperand<T>{G, kE, c.T * kE, int(c.T), n8}
                                            : DenseOperand<T>{G, h.ldg, kE, int(c.T), n8};
      const DenseOperand<T> B =
          c.by_vocab ? DenseOperand<T>{a.W.p, h.ldw, 0, int(round8(c.H)), int(n)}
                     : DenseOperand<T>{a.W.p, h.ldw, kE, int(c.H), n8};
      const int64_t per = ceil_div(ceil_div(n, h.slices), 64) * 64;
      if (direct) {
        const ProductArgs<T, T> q{A, B, int(c.T), int(c.H), n8, static_cast<T*>(c.dX), c.lddx, 0, 1,
                                  c.top};
        e = c.by_vocab ? product<T, kAlong, kAcross, T, false>(tx, q, 1, stream)
                       : product<T, kAlong, kAlong, T, false>(tx, q, 1, stream);
      } else {
        const ProductArgs<T, float> q{A, B, int(c.T), int(c.H), int(per), c.acc, h.ldp,
                                      c.T * h.ldp, v0 == 0, nullptr};
        e = c.by_vocab ? product<T, kAlong, kAcross, float, true>(tx, q, h.slices, stream)
                       : product<T, kAlong, kAlong, float, true>(tx, q, h.slices, stream);
      }
      if (e != hipSuccess) return e;
    }
    // dW's piece: X^T G (H x n) or G^T X (n x H), reduction over the rows
    const int64_t rows = c.by_vocab ? n : c.H, cols = c.by_vocab ? c.H : n;
    constexpr int kAcrossRows = kGPieces<T> ? kPieces : kAcross;
    const DenseOperand<T> Gt = kGPieces<T>
                                   ? DenseOperand<T>{G, 0, c.T * 32, int(round32(n)), int(c.T)}
                                   : DenseOperand<T>{G, h.ldg, 0, n8, int(c.T)};
    const DenseOperand<T> Xt =
        kGPieces<T> ? DenseOperand<T>{X.p, 0, c.T * 32, int(round32(c.H)), int(c.T)}
                    : DenseOperand<T>{X.p, X.ld, 0, int(round8(c.H)), int(c.T)};
    const ProductArgs<T, T> q{c.by_vocab ? Gt : Xt, c.by_vocab ? Xt : Gt, int(rows), int(cols),
                              int(c.T), dW + v0 * (c.by_vocab ? c.lddw : 1), c.lddw, 0, 1, c.top};
    e = product<T, kAcrossRows, kAcrossRows, T, false>(pick_tile(kBf16, rows, cols), q, 1, stream);
    if (e != hipSuccess) return e;
  }
  if (direct || c.T == 0) return hipSuccess;
  head_sum_kernel<T><<<copy_blocks(c.T * (h.ldp / 4)), 256, 0, stream>>>(
      c.acc, int(h.slices), c.T * h.ldp, c.T, int(c.H), h.ldp, c.top, static_cast<T*>(c.dX),
      c.lddx);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_head_loss(const HeadCall& c, bool bf16, const HeadPlan& h, hipStream_t stream) {
  return bf16 ? run_forward<uint16_t>(c, h, stream) : run_forward<float>(c, h, stream);
}

hipError_t launch_head_loss_backward(const HeadCall& c, bool bf16, const HeadPlan& h,
                                     hipStream_t stream) {
  return bf16 ? run_backward<uint16_t>(c, h, stream) : run_backward<float>(c, h, stream);
}

}  // namespace fp4lin
