// Products grouped by expert on micro-scaled FP4 operands.
//
// The rows of the activations are sorted by expert: expert e owns the rows
// [b_e, n_e), n_e = row_end[e] and b_e = n_(e-1) (b_0 = 0), in numbers that only
// the device knows. With Q the block quantization of mx.hip along the product's
// reduction,
//   forward  Y[r, :]  = Q(A)[r, :] . Q(W[e])        over K, for the rows r of e
//   dgrad    dX[r, :] = Q(dY)[r, :] . Q(W[e])^T     over N
//   wgrad    dW[e]    = Q(A_e)^T . Q(dY_e)          over e's rows; blocks of 32
//                                                   rows count from its first row
// Each is a sum over blocks of 2^(eA + eB) * (FP4 dot product), accumulated in
// fp32 by the matrix core and written once, in fp32 or rounded to bfloat16. A block
// that holds an infinity or NaN has the scale NaN in every form of the products
// (BlockMax), so that none of them turns one into a number.
//
// Ragged groups without a host copy of row_end: a launch covers the most tiles
// that any split of the rows over the experts can need, every wave finds its
// tile's expert by a scan over row_end (64 experts a round: one load, a running
// maximum and a prefix sum across lanes), and workgroups past the last tile
// end at once. The scan also gives the number of tiles, which the mapping of
// workgroups to XCDs needs. row_end is read as a running maximum clamped to
// [0, M], so no content of it can lead outside the operands.
//
// Rows at and past the last expert's end belong to nobody: their output rows
// are written as zeros by the workgroups of one more group.
#include <type_traits>

#include "colquant.hpp"
#include "device_common.hpp"
#include "gemm_core.hpp"
#include "internal.hpp"

namespace fp4lin {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Groups.
// ---------------------------------------------------------------------------
// Running maximum and sum across the wave (inclusive) of values >= 0, on the
// vector unit: shifts within rows of 16 lanes (lanes without a source take 0),
// then the last lane of a row to the next row and of the first half to the second.
template <class Op>
__device__ inline int wave_scan(int v, const Op& op) {
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // row_shr:1
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // row_bcast:15
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // row_bcast:31
  return v;
}
__device__ inline int wave_scan_max(int v) {
  return wave_scan(v, [](int a, int b) { return a > b ? a : b; });
}
__device__ inline int wave_scan_sum(int v) {
  return wave_scan(v, [](int a, int b) { return a + b; });
}

// A group of rows: expert e's, or with e == E the rows past the last expert's
// end. first: the units (of R rows, the last one of a group part full) of all
// groups before it.
struct Group {
  int e, begin, rows, first;
};

// 64 experts of the scan, one per lane: [begin, end) and the units up to and
// with the lane's own. Lanes past E hold empty groups.
template <int R>
struct GroupScan {
  int begin, end, upto;

  __device__ inline void read(const int32_t* row_end, int base, int E, int M, int end0,
                              int units0) {
    const int lane = threadIdx.x & (kWave - 1);
    int n = base + lane < E ? row_end[base + lane] : 0;
    n = n < 0 ? 0 : (n > M ? M : n);
    n = wave_scan_max(n > end0 ? n : end0);
    const int p = __shfl_up(n, 1, kWave);
    begin = lane == 0 ? end0 : p;
    end = n;
    upto = units0 + wave_scan_sum((end - begin + R - 1) / R);
  }
  __device__ inline Group group(int base, int lane) const {
    const int b = __builtin_amdgcn_readlane(begin, lane);
    const int n = __builtin_amdgcn_readlane(end, lane);
    const int u = __builtin_amdgcn_readlane(upto, lane);
    return Group{base + lane, b, n - b, u - (n - b + R - 1) / R};
  }
};

// The group of unit pick(total), total the number of units of all groups, the one
// past the last expert among them; pick may answer none (negative): then e < 0.
// Up to 64 experts are scanned once, more twice.
template <int R, class Pick>
__device__ inline Group group_of_unit(const int32_t* row_end, int E, int M, const Pick& pick) {
  GroupScan<R> first;
  first.read(row_end, 0, E, M, 0, 0);
  int end = __builtin_amdgcn_readlane(first.end, kWave - 1);
  int units = __builtin_amdgcn_readlane(first.upto, kWave - 1);
  for (int base = kWave; base < E; base += kWave) {
    GroupScan<R> s;
    s.read(row_end, base, E, M, end, units);
    end = __builtin_amdgcn_readlane(s.end, kWave - 1);
    units = __builtin_amdgcn_readlane(s.upto, kWave - 1);
  }
  const int u = pick(units + (M - end + R - 1) / R);
  if (u < 0) return Group{-1, 0, 0, 0};
  if (u >= units) return Group{E, end, M - end, units};
  uint64_t past = __ballot(u < first.upto);
  int base = 0;
  while (past == 0) {
    const int end0 = __builtin_amdgcn_readlane(first.end, kWave - 1);
    const int units0 = __builtin_amdgcn_readlane(first.upto, kWave - 1);
    base += kWave;
    first.read(row_end, base, E, M, end0, units0);
    past = __ballot(u < first.upto);
  }
  return first.group(base, __builtin_ctzll(past));
}

// Group e (0 <= e <= E).
template <int R>
__device__ inline Group group_of_expert(const int32_t* row_end, int E, int M, int e) {
  int end0 = 0, units0 = 0;
  for (int base = 0; base < E; base += kWave) {
    GroupScan<R> s;
    s.read(row_end, base, E, M, end0, units0);
    if (e < base + kWave && e < E) return s.group(base, e - base);
    end0 = __builtin_amdgcn_readlane(s.end, kWave - 1);
    units0 = __builtin_amdgcn_readlane(s.upto, kWave - 1);
  }
  return Group{E, end0, M - end0, units0};
}

// ---------------------------------------------------------------------------
// Quantizers. Operands that only a product of this file reads are kept with the
// codes of a K step together (Fp4Operand), rows of one matrix or expert at a
// time; the two operands of a product are quantized in one launch, whose first
// workgroups take the first one.
// ---------------------------------------------------------------------------
struct RowsArgs {
  const void* X;
  int64_t M, L, ldx;  // rows, reduction
  int64_t block;      // rows whose codes of a step are together
  uint8_t *q, *s;
  int gx, gy;         // workgroups
};

struct ColsArgs {
  const void* W;
  int64_t E, K, N, ldw;
  int64_t ld, step;  // of the codes (quantize_cols_mx_body), within an expert
  uint8_t *q, *s;
  int gx, gy;  // workgroups of an expert
};

template <class In, bool kFast, int kRows>
__device__ inline void quantize_rows_part(const RowsArgs& p, int id) {
  quantize_rows_mx_body<In, kFast, kRows, true>(
      id % p.gx, p.gx, id / p.gx, p.gy, static_cast<const typename In::T*>(p.X), p.M, p.L, p.ldx,
      __builtin_huge_valf(), p.q, (p.L + 127) / 128 * 64, p.block, p.s);
}

// Rows of two matrices (dgrad: dY and the weights; apply: the activations alone).
// Bound by memory: 16 experts 2048 x 5632 and 8192 rows 122 us for 461 MB read and
// 122 MB written (4.8 TB/s).
template <class In, bool kFast, int kRows>
__global__ __launch_bounds__(kThreads) void experts_rows_mx_kernel(RowsArgs a, RowsArgs b) {
  const int id = blockIdx.x, na = a.gx * a.gy;
  if (id < na)
    quantize_rows_part<In, kFast, kRows>(a, id);
  else
    quantize_rows_part<In, kFast, kRows>(b, id - na);
}

// Weights along K (rows of W[e]), a 128 x 128 tile a workgroup; with kRows > 0
// rows of the activations first. Scales go to one step-major array over the E * N
// columns of all experts. Bound by memory: 8 experts 4096 x 11008 and 8192 rows 192
// us for 788 MB read and 209 MB written (5.2 TB/s, as a copy).
template <class In, bool kFast, int kRows>
__global__ __launch_bounds__(kThreads) void experts_cols_mx_kernel(RowsArgs a, ColsArgs w) {
  int id = blockIdx.x;
  if constexpr (kRows > 0) {
    const int na = a.gx * a.gy;
    if (id < na) {
      quantize_rows_part<In, kFast, kRows>(a, id);
      return;
    }
    id -= na;
  }
  const int64_t e = id / (w.gx * w.gy);
  id -= int(e) * w.gx * w.gy;
  quantize_cols_mx_body<In, kFast, true>(
      id % w.gx, id / w.gx, static_cast<const typename In::T*>(w.W) + e * w.K * w.ldw, w.K, w.N,
      w.ldw, w.q + e * w.N * ((w.K + 127) / 128 * 64), w.ld, w.step, w.s + 4 * e * w.N, w.E * w.N);
}

// Activations and gradients along each expert's own rows: K step blockIdx.y of
// all experts' steps (128 rows each, the last one of an expert filled with zeros)
// and 128 columns of A (K of them) or, past those, of dY (N). 60 us for 247 MB read
// and 66 MB written (8192 rows, 4096 and 11008 columns; 5.2 TB/s).
struct RaggedArgs {
  const void *A, *dY;
  const int32_t* row_end;
  int E, M, K, N;
  int64_t lda, lddy;
  uint8_t *Aq, *As, *Dq, *Ds;
};

template <class In, bool kAligned>
__global__ __launch_bounds__(kThreads) void experts_ragged_mx_kernel(RaggedArgs p) {
  using T = typename In::T;
  const int s = blockIdx.y;
  const Group g =
      group_of_unit<128>(p.row_end, p.E, p.M, [&](int total) { return s < total ? s : -1; });
  if (g.e < 0 || g.e == p.E) return;
  const int tiles = (p.K + kMxTN - 1) / kMxTN;
  const bool first = int(blockIdx.x) < tiles;
  const int64_t n = first ? p.K : p.N, ld = first ? p.lda : p.lddy;
  quantize_cols_mx_body<In, kAligned, true>(
      first ? blockIdx.x : blockIdx.x - tiles, s - g.first,
      static_cast<const T*>(first ? p.A : p.dY) + int64_t(g.begin) * ld, g.rows, n, ld,
      (first ? p.Aq : p.Dq) + int64_t(g.first) * 64 * n, 64, 64 * n,
      (first ? p.As : p.Ds) + int64_t(g.first) * 4 * n, n);
}

// ---------------------------------------------------------------------------
// Products over tiles.
// ---------------------------------------------------------------------------
struct TileArgs {
  const uint8_t *Aq, *As, *Bq, *Bs;
  const int32_t* row_end;
  int E, M;        // M: rows of the activations
  int rows, cols;  // of an expert's output (rows: wgrad only)
  int ldq;         // bytes of a packed row (wgrad: of all experts' steps)
  int packed;      // B in packed rows, not a step's rows together
  void* Y;
  int64_t ldy;
};

// Bound by what the tiles write and by the matrix core in turn, as a 256 x 256 tile
// has a CU to itself. Launched alone, one after the other: the product of the forward
// of 8192 rows, 8 experts 4096 x 11008, 218 us (3.4 PFLOP/s); without its stores (361
// MB of fp32) 174 us, 4.2 PFLOP/s (the instruction stream alone reaches 5.7), without
// its loop 72. The wgrad there has four or five K steps a tile and writes 1.44 GB: 390
// us, 248 without the stores, 281 without the loop. (Under the profiler, at lower
// clocks, 285 and 387.)
//
// kWgrad false: forward and dgrad, A the rows of the activations, B the weights
// of all experts (cols rows each). kWgrad true: A and B the columns of the
// activations and gradients, expert e's steps a range of the steps of both.
template <class C, class Out, bool kWgrad>
__global__ __launch_bounds__(C::kThreads, C::kMinBlocks) void experts_gemm_kernel(TileArgs p) {
  constexpr int SB = C::kStageBytes;
  __shared__ __attribute__((aligned(16))) uint8_t st0[SB];
  __shared__ __attribute__((aligned(16))) uint8_t st1[SB];
  __shared__ __attribute__((aligned(16))) uint8_t st2[SB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.cols + C::BN - 1) / C::BN;
  int m0, n0, rows, nkt;
  Fp4Operand A, B;
  Out* Y = static_cast<Out*>(p.Y);
  if constexpr (kWgrad) {
    const int tiles_m = (p.rows + C::BM - 1) / C::BM;
    const int t = xcd_run(blockIdx.x, p.E * tiles_m * tiles_n);
    if (t < 0) return;
    const int e = t / (tiles_m * tiles_n);
    int tm, tn;
    tile_of(t - e * tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
    const Group g = group_of_expert<128>(p.row_end, p.E, p.M, e);
    nkt = (g.rows + 127) / 128;
    m0 = tm * C::BM;
    n0 = tn * C::BN;
    rows = p.rows;
    const int64_t s = g.first;
    A = Fp4Operand{p.Aq + s * 64 * p.rows, 64, 64 * p.rows, p.rows, nkt * 64 * p.rows,
                   p.As + s * 4 * p.rows, 4 * p.rows, nkt * 4 * p.rows};
    B = Fp4Operand{p.Bq + s * 64 * p.cols, 64, 64 * p.cols, p.cols, nkt * 64 * p.cols,
                   p.Bs + s * 4 * p.cols, 4 * p.cols, nkt * 4 * p.cols};
    Y += int64_t(e) * p.rows * p.ldy;
  } else {
    int t = -1;
    const Group g = group_of_unit<C::BM>(p.row_end, p.E, p.M, [&](int total) {
      t = xcd_run(blockIdx.x, total * tiles_n);
      return t < 0 ? -1 : t / tiles_n;
    });
    if (g.e < 0) return;
    int tm, tn;
    tile_of(t - g.first * tiles_n, (g.rows + C::BM - 1) / C::BM, tiles_n, tm, tn);
    // the rows past the last expert's end: no steps, zeros
    nkt = g.e == p.E ? 0 : p.ldq / 64;
    m0 = tm * C::BM;
    n0 = tn * C::BN;
    rows = g.rows;
    const int nblk = p.ldq / 16, all = p.E * p.cols, e = g.e == p.E ? 0 : g.e;
    A = Fp4Operand{p.Aq + int64_t(g.begin) * 64, 64, p.M * 64, g.rows, p.M * p.ldq - g.begin * 64,
                   p.As + 4 * int64_t(g.begin), 4 * p.M, p.M * nblk - 4 * g.begin};
    B = Fp4Operand{p.Bq + int64_t(e) * p.cols * p.ldq, p.packed ? p.ldq : 64,
                   p.packed ? 64 : 64 * p.cols, p.cols, p.cols * p.ldq,
                   p.Bs + 4 * int64_t(e) * p.cols, 4 * all, all * nblk - 4 * e * p.cols};
    Y += int64_t(g.begin) * p.ldy;
  }
  Fp4Feed<C, true> f(A, B, m0, n0, wave, lane);
  if (nkt > 0) gemm_pipeline(f, nkt, st0, st1, st2);
  store_tile<C>(st0, st1, st2, wave, lane, m0, n0, rows, p.cols, Y, p.ldy,
                [&](int fm, int fn, int r) { return f.acc[fm][fn][r]; });
}

// ---------------------------------------------------------------------------
// A few rows in all (serving one or some tokens): bound by latency and by
// reading the weights' codes once, in one launch.
// ---------------------------------------------------------------------------
// A workgroup of W waves owns 16 columns of one expert. The waves split K: wave
// w takes the K steps w, w + W, ..., at most kSteps of them, so that the waves
// read contiguous bytes of each column's packed row. Codes go from memory
// straight to the matrix core's registers (the 16x16x128 shape: lane l holds the
// 32 codes of block l / 16 of the step for column l % 16, one 16-byte load, and
// the block's scale byte). While they are on their way the workgroup quantizes
// its expert's rows into LDS: at this size that costs less than a launch of its
// own would (one token, two of 8 experts 2048x5632: 11.0 against 14.2 us a call, 6.5
// of them on the GPU for 12.3 MB of codes: latency, one load deep).
// The waves' partial sums are added in wave order through LDS.
constexpr int kSteps = 8;
constexpr int64_t kFusedRows = 16, kFusedElems = 8192;  // of the activations

typedef float v4f __attribute__((ext_vector_type(4)));

struct FewArgs {
  const void* A;  // M x K
  int64_t lda;
  int fast;  // A allows 16-byte loads of 8 elements
  const uint8_t *Bq, *Bs;
  const int32_t* row_end;
  int E, M, K, N, ldq;
  void* Y;
  int64_t ldy;
};

__device__ inline void store_out(float* p, float v) { *p = v; }
__device__ inline void store_out(uint16_t* p, float v) { *p = uint16_t(bf16_pair(v, v)); }

// Rows begin .. begin + rows - 1 of A as codes (ldq bytes a row) and scale
// bytes (ldq / 16 a row) in LDS.
template <class In>
__device__ inline void quantize_few(const FewArgs& p, int begin, int rows, uint8_t* codes,
                                    uint8_t* scales) {
  const int cpr = p.ldq / 4;  // chunks of 8 codes a row; four lanes hold a block
  for (int i = threadIdx.x; i < rows * cpr; i += blockDim.x) {
    const int r = i / cpr, c = i - r * cpr;
    const auto* row = static_cast<const typename In::T*>(p.A) + (begin + r) * p.lda;
    Vec8<In> v;
    if (p.fast)
      load_chunk<In, true>(row, c * 8, p.K, v);
    else
      load_chunk<In, false>(row, c * 8, p.K, v);
    float ax[8];
    BlockMax<true> m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ax[j] = fabsf(In::widen(v.v[j]));
      m.take(ax[j]);
    }
    const int e = m.exponent();
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      word |= (mx_magnitude(ax[j], e) | (In::sign_bit(v.v[j]) << 3)) << (4 * j);
    *reinterpret_cast<uint32_t*>(codes + r * p.ldq + c * 4) = word;
    if ((c & 3) == 0) scales[r * (p.ldq / 16) + c / 4] = uint8_t(e + 127);
  }
}

template <int W, class In, class Out>
__global__ __launch_bounds__(W * 64) void experts_few_kernel(FewArgs p) {
  __shared__ v4f part[W][64];
  // at most kFusedRows rows of M * K <= kFusedElems elements, each padded
  constexpr int kCodeBytes = kFusedElems / 2 + kFusedRows * 64;
  __shared__ __attribute__((aligned(16))) uint8_t codes[kCodeBytes];
  __shared__ uint8_t scales[kCodeBytes / 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Group g = group_of_expert<16>(p.row_end, p.E, p.M, blockIdx.y);
  if (g.rows == 0) return;
  Out* const Y = static_cast<Out*>(p.Y);
  const int n = blockIdx.x * 16 + (lane & 15);
  const int q = lane >> 4;
  v4f acc{};
  if (g.e < p.E) {
    const int nkt = p.ldq / 64;
    const int64_t bcol = int64_t(g.e) * p.N + (n < p.N ? n : p.N - 1);
    const int64_t bstep = 4 * int64_t(p.E) * p.N;
    uint4 b[kSteps];
    int sb[kSteps], at[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      // steps past the end repeat the last one and are not multiplied
      const int s = wave + u * W < nkt ? wave + u * W : nkt - 1;
      at[u] = s;
      b[u] = *reinterpret_cast<const uint4*>(p.Bq + bcol * p.ldq + s * 64 + q * 16);
      sb[u] = p.Bs[s * bstep + 4 * bcol + q];
    }
    quantize_few<In>(p, g.begin, g.rows, codes, scales);
    __syncthreads();
    // rows past the group's end repeat its last row; they are not stored
    const int ra = (lane & 15) < g.rows ? (lane & 15) : g.rows - 1;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      if (wave + u * W >= nkt) break;
      const uint4 a = *reinterpret_cast<const uint4*>(codes + ra * p.ldq + at[u] * 64 + q * 16);
      const int sa = scales[ra * (p.ldq / 16) + at[u] * 4 + q];
      const v8i af{int(a.x), int(a.y), int(a.z), int(a.w), 0, 0, 0, 0};
      const v8i bf{int(b[u].x), int(b[u].y), int(b[u].z), int(b[u].w), 0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af, bf, acc, 4, 4, 0, sa, 0, sb[u]);
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  v4f sum = part[0][lane];
#pragma unroll
  for (int w = 1; w < W; ++w) sum += part[w][lane];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int r = 4 * q + c;
    if (r < g.rows && n < p.N) store_out(Y + (g.begin + r) * p.ldy + n, sum[c]);
  }
}

using LargeTile = GemmCfg<256, 256, 4, 2, 64, 1>;
using SmallTile = GemmCfg<128, 256, 2, 2, 64, 2>;
using FewTile = GemmCfg<64, 128, 1, 2, 64, 2>;
constexpr int64_t kLargeTilesMin = 512;
constexpr int64_t kSmallTilesMin = 256;
constexpr int64_t kFewRows = 32;  // rows an expert on average

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class C, class Out, bool kWgrad>
hipError_t run_tiles(const TileArgs& p, int64_t tiles, hipStream_t stream) {
  if (tiles >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  experts_gemm_kernel<C, Out, kWgrad><<<dim3(unsigned(tiles)), C::kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

// Row tiles of BM rows that M rows in at most E + 1 groups can need.
int64_t most_units(int64_t M, int64_t E, int64_t R) {
  const int64_t groups = E + 1 < M ? E + 1 : M;
  return (M + groups * (R - 1)) / R;
}

template <class In, class Out>
hipError_t run_few(const FewArgs& a, hipStream_t stream) {
  const dim3 grid(unsigned(ceil_div(a.N, 16)), unsigned(a.E + 1));
  static_assert(kFusedElems <= 8 * kSteps * 128, "eight waves hold K");
  if (a.ldq / 64 <= 4 * kSteps)
    experts_few_kernel<4, In, Out><<<grid, 4 * 64, 0, stream>>>(a);
  else
    experts_few_kernel<8, In, Out><<<grid, 8 * 64, 0, stream>>>(a);
  return hipGetLastError();
}

// Tiles of 256 x 256 where they fill the CUs twice, of 128 x 256 where those
// fill them once, else of 64 x 128; the last also for few rows an expert, where
// a product is a read of the weights' codes and more workgroups on their way
// read faster (8 experts 4096x11008, whole call: 128 rows 47 against 53 us with
// 128 x 256 tiles, 256 rows 51 against 57, 512 rows 60 against 62). Whole calls with 256 x
// 256 / 128 x 256 / 64 x 128 tiles alone: forward of 8192 rows, 8 experts 4096x11008
// 429 / 437 / 488 us, of 2048 rows 275 / 261 / 284, of 1024 rows, 8 experts 2048x5632
// 61 / 64 / 62, of 8192 rows, 16 experts 189 / 198 / 221 and 64 experts (whose large
// tiles are half empty) 509 / 494 / 511; dgrad of 8192 rows, 16 experts 202 / 195 / 212.
template <class Out>
hipError_t run_rows(const TileArgs& p, hipStream_t stream) {
  const int64_t tiles_n = ceil_div(p.cols, 256);
  if (ceil_div(p.M, LargeTile::BM) * tiles_n >= kLargeTilesMin)
    return run_tiles<LargeTile, Out, false>(p, most_units(p.M, p.E, LargeTile::BM) * tiles_n,
                                            stream);
  if (p.M > kFewRows * p.E && ceil_div(p.M, SmallTile::BM) * tiles_n >= kSmallTilesMin)
    return run_tiles<SmallTile, Out, false>(p, most_units(p.M, p.E, SmallTile::BM) * tiles_n,
                                            stream);
  return run_tiles<FewTile, Out, false>(
      p, most_units(p.M, p.E, FewTile::BM) * ceil_div(p.cols, FewTile::BN), stream);
}

// The same choice: 4096 rows, 8 experts 1024x2816 42 us with 256 x 256 tiles, 39 with
// 128 x 256 (352 large tiles); 16384 rows, 4 experts 2048x5632 211 and 217. (8192 rows,
// 8 experts 4096x11008, with few K steps a tile: 454 and 438, on another card 434 and 430.)
template <class Out>
hipError_t run_wgrad(const TileArgs& p, hipStream_t stream) {
  const int64_t tiles_n = ceil_div(p.cols, 256);
  const int64_t large = p.E * ceil_div(p.rows, LargeTile::BM) * tiles_n;
  if (large >= kLargeTilesMin) return run_tiles<LargeTile, Out, true>(p, large, stream);
  return run_tiles<SmallTile, Out, true>(p, p.E * ceil_div(p.rows, SmallTile::BM) * tiles_n,
                                         stream);
}

bool rows_fast(const void* X, int64_t ldx, int64_t L, int bytes) {
  return reinterpret_cast<uintptr_t>(X) % 16 == 0 && (ldx * bytes) % 16 == 0 && L % 8 == 0;
}
bool cols_fast(const void* X, int64_t ldx, int bytes) {
  return reinterpret_cast<uintptr_t>(X) % 16 == 0 && (ldx * bytes) % 16 == 0;
}

void rows_grid(RowsArgs& a, int rows) {
  if (a.M == 0) return;
  const dim3 g = mx_row_grid(a.M, (a.L + 127) / 128 * 16, rows);
  a.gx = int(g.x);
  a.gy = int(g.y);
}
bool many(const RowsArgs& a) { return a.M * ((a.L + 127) / 128 * 64) >= kManyRowBytes; }

// One or two (b.M > 0) matrices by rows.
template <class In>
hipError_t run_rows_mx(RowsArgs a, RowsArgs b, hipStream_t stream) {
  const bool fast = rows_fast(a.X, a.ldx, a.L, In::kBytes) &&
                    (b.M == 0 || rows_fast(b.X, b.ldx, b.L, In::kBytes));
  const int rows = fast && (many(a) || many(b)) ? 4 : 1;
  rows_grid(a, rows);
  rows_grid(b, rows);
  const unsigned grid = unsigned(a.gx) * unsigned(a.gy) + unsigned(b.gx) * unsigned(b.gy);
  if (rows == 4)
    experts_rows_mx_kernel<In, true, 4><<<grid, kThreads, 0, stream>>>(a, b);
  else if (fast)
    experts_rows_mx_kernel<In, true, 1><<<grid, kThreads, 0, stream>>>(a, b);
  else
    experts_rows_mx_kernel<In, false, 1><<<grid, kThreads, 0, stream>>>(a, b);
  return hipGetLastError();
}

// The weights along K, and (a.M > 0) rows of the activations.
template <class In>
hipError_t run_cols_mx(RowsArgs a, ColsArgs w, hipStream_t stream) {
  const bool fast =
      cols_fast(w.W, w.ldw, In::kBytes) && (a.M == 0 || rows_fast(a.X, a.ldx, a.L, In::kBytes));
  const int rows = fast && many(a) ? 4 : 1;
  rows_grid(a, rows);
  w.gx = int(ceil_div(w.N, kMxTN));
  w.gy = int(ceil_div(w.K, kMxTK));
  const unsigned grid = unsigned(a.gx) * unsigned(a.gy) + unsigned(w.E * w.gx * w.gy);
  if (a.M == 0) {
    if (fast)
      experts_cols_mx_kernel<In, true, 0><<<grid, kThreads, 0, stream>>>(a, w);
    else
      experts_cols_mx_kernel<In, false, 0><<<grid, kThreads, 0, stream>>>(a, w);
  } else if (rows == 4) {
    experts_cols_mx_kernel<In, true, 4><<<grid, kThreads, 0, stream>>>(a, w);
  } else if (fast) {
    experts_cols_mx_kernel<In, true, 1><<<grid, kThreads, 0, stream>>>(a, w);
  } else {
    experts_cols_mx_kernel<In, false, 1><<<grid, kThreads, 0, stream>>>(a, w);
  }
  return hipGetLastError();
}

template <class In>
hipError_t run_ragged(const RaggedArgs& p, int64_t steps, hipStream_t stream) {
  const dim3 grid(unsigned(ceil_div(p.K, kMxTN) + ceil_div(p.N, kMxTN)), unsigned(steps));
  if (cols_fast(p.A, p.lda, In::kBytes) && cols_fast(p.dY, p.lddy, In::kBytes))
    experts_ragged_mx_kernel<In, true><<<grid, kThreads, 0, stream>>>(p);
  else
    experts_ragged_mx_kernel<In, false><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

int64_t experts_steps(int64_t E, int64_t M) {
  const int64_t groups = E < M ? E : M;
  return (M + groups * 127) / 128;
}

hipError_t launch_experts_quantize_weight_mx(const void* W, bool bf16, int64_t E, int64_t K,
                                             int64_t N, int64_t ldw, uint8_t* Wq, int64_t ldq,
                                             uint8_t* Ws, hipStream_t stream) {
  const ColsArgs w{W, E, K, N, ldw, ldq, 64, Wq, Ws, 0, 0};
  return bf16 ? run_cols_mx<BF16In>(RowsArgs{}, w, stream) : run_cols_mx<F32In>(RowsArgs{}, w, stream);
}

hipError_t launch_experts_quantize_forward(const void* A, const void* W, bool bf16, int64_t E,
                                           int64_t M, int64_t K, int64_t N, int64_t lda,
                                           int64_t ldw, uint8_t* Aq, uint8_t* As, uint8_t* Wq,
                                           uint8_t* Ws, hipStream_t stream) {
  const RowsArgs a{A, M, K, lda, M, Aq, As, 0, 0};
  const ColsArgs w{W, E, K, N, ldw, 64, 64 * N, Wq, Ws, 0, 0};
  return bf16 ? run_cols_mx<BF16In>(a, w, stream) : run_cols_mx<F32In>(a, w, stream);
}

hipError_t launch_experts_quantize_rows(const void* A, bool bf16, int64_t M, int64_t K, int64_t lda,
                                        uint8_t* Aq, uint8_t* As, hipStream_t stream) {
  const RowsArgs a{A, M, K, lda, M, Aq, As, 0, 0};
  return bf16 ? run_rows_mx<BF16In>(a, RowsArgs{}, stream) : run_rows_mx<F32In>(a, RowsArgs{}, stream);
}

hipError_t launch_experts_quantize_dgrad(const void* dY, const void* W, bool bf16, int64_t E,
                                         int64_t M, int64_t K, int64_t N, int64_t lddy, int64_t ldw,
                                         uint8_t* Dq, uint8_t* Ds, uint8_t* Wq, uint8_t* Ws,
                                         hipStream_t stream) {
  const RowsArgs a{dY, M, N, lddy, M, Dq, Ds, 0, 0};
  const RowsArgs w{W, E * K, N, ldw, K, Wq, Ws, 0, 0};
  return bf16 ? run_rows_mx<BF16In>(a, w, stream) : run_rows_mx<F32In>(a, w, stream);
}

hipError_t launch_experts_quantize_wgrad(const void* A, const void* dY, bool bf16,
                                         const int32_t* row_end, int64_t E, int64_t M, int64_t K,
                                         int64_t N, int64_t lda, int64_t lddy, uint8_t* Aq,
                                         uint8_t* As, uint8_t* Dq, uint8_t* Ds,
                                         hipStream_t stream) {
  const int64_t steps = experts_steps(E, M);
  if (steps == 0) return hipSuccess;
  const RaggedArgs p{A, dY, row_end, int(E), int(M), int(K), int(N), lda, lddy, Aq, As, Dq, Ds};
  return bf16 ? run_ragged<BF16In>(p, steps, stream) : run_ragged<F32In>(p, steps, stream);
}

hipError_t launch_experts_rows(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                               const uint8_t* Bs, const int32_t* row_end, int64_t E, int64_t M,
                               int64_t N, int64_t ldq, bool packed, void* Y, bool y_bf16,
                               int64_t ldy, hipStream_t stream) {
  const TileArgs p{Aq, As, Bq, Bs, row_end, int(E), int(M), 0, int(N), int(ldq), packed, Y, ldy};
  return y_bf16 ? run_rows<uint16_t>(p, stream) : run_rows<float>(p, stream);
}

bool experts_fused(int64_t M, int64_t K) { return M <= kFusedRows && M * K <= kFusedElems; }

hipError_t launch_experts_fused(const void* A, bool bf16, int64_t lda, const uint8_t* Bq,
                                const uint8_t* Bs, const int32_t* row_end, int64_t E, int64_t M,
                                int64_t K, int64_t N, int64_t ldq, void* Y, bool y_bf16,
                                int64_t ldy, hipStream_t stream) {
  FewArgs a{};
  a.A = A;
  a.lda = lda;
  a.fast = reinterpret_cast<uintptr_t>(A) % 16 == 0 && (lda * (bf16 ? 2 : 4)) % 16 == 0 && K % 8 == 0;
  a.Bq = Bq;
  a.Bs = Bs;
  a.row_end = row_end;
  a.E = int(E);
  a.M = int(M);
  a.K = int(K);
  a.N = int(N);
  a.ldq = int(ldq);
  a.Y = Y;
  a.ldy = ldy;
  if (bf16)
    return y_bf16 ? run_few<BF16In, uint16_t>(a, stream) : run_few<BF16In, float>(a, stream);
  return y_bf16 ? run_few<F32In, uint16_t>(a, stream) : run_few<F32In, float>(a, stream);
}

hipError_t launch_experts_wgrad(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                                const uint8_t* Bs, const int32_t* row_end, int64_t E, int64_t M,
                                int64_t K, int64_t N, void* dW, bool w_bf16, int64_t ldw,
                                hipStream_t stream) {
  const TileArgs p{Aq, As, Bq, Bs, row_end, int(E), int(M), int(K), int(N),
                   int(experts_steps(E, M) * 64), 0, dW, ldw};
  return w_bf16 ? run_wgrad<uint16_t>(p, stream) : run_wgrad<float>(p, stream);
}

}  // namespace fp4lin
