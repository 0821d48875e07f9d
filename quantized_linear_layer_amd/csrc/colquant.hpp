// Channel-wise (per column) quantization of a K x N row-major matrix into
// E2M1 codes packed N-major, as device bodies of 256-thread workgroups that
// take their workgroup coordinates as arguments: the column-max pass and the
// encode pass of the token-wise format, and the one pass of the micro-scaled
// format (blocks of 32 codes along K); and the row pass of the micro-scaled format.
// The quantize_weight kernels launch
// them directly; the forward pairs them with the select's row kernels in
// shared launches.
#pragma once

#include "device_common.hpp"

namespace fp4lin {

constexpr int kColStrip = 512;    // columns per workgroup (8 per lane)
constexpr int kColRows = 64;      // rows per workgroup split
constexpr int kColUnroll = 8;     // loads in flight per thread

// Pass 1, workgroup (bx, by): columns bx*512 .. +511, rows by*64 .. +63.
template <class In, bool kAligned>
__device__ __attribute__((always_inline)) inline void colmax_body(int64_t bx, int64_t by, const typename In::T* __restrict__ W,
                                   int64_t K, int64_t N, int64_t ldw,
                                   uint32_t* __restrict__ colmax) {
  __shared__ uint32_t red[4][kColStrip];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int64_t c = bx * kColStrip + lane * 8;
  const int64_t k0 = by * kColRows;
  const int64_t k1 = (k0 + kColRows < K) ? k0 + kColRows : K;
  const int64_t valid = N - c;
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = 0.0f;
  if (valid > 0) {
    // kColUnroll rows in flight per thread; rows past k1 read as zero
    for (int64_t kb = k0 + wave; kb < k1; kb += 4 * kColUnroll) {
      Vec8<In> v[kColUnroll];
#pragma unroll
      for (int u = 0; u < kColUnroll; ++u) {
        const int64_t k = kb + 4 * u;
        if (k < k1) {
          load8<In, kAligned>(W + k * ldw + c, valid, v[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u].v[i] = typename In::T(0);
        }
      }
#pragma unroll
      for (int u = 0; u < kColUnroll; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], fabsf(In::widen(v[u].v[i])));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[wave][lane * 8 + i] = __float_as_uint(m[i]);
  __syncthreads();
  for (int j = threadIdx.x; j < kColStrip; j += 256) {
    uint32_t x = red[0][j];
    x = x > red[1][j] ? x : red[1][j];
    x = x > red[2][j] ? x : red[2][j];
    x = x > red[3][j] ? x : red[3][j];
    const int64_t col = bx * kColStrip + j;
    if (col < N) atomicMax(&colmax[col], x);
  }
}

// Pass 2 tile: 128 codes along K x 128 columns. Thread (kg, g) = (t % 16,
// t / 16) owns rows k0 + 8kg .. +7 and columns n0 + 8g .. +7, so for each of its
// columns the 8 codes along K form one 32-bit word of that column's packed row
// (low nibble first), stored directly: a wave's store covers 64 contiguous
// bytes of each of 4 packed rows, and its loads 64 contiguous bytes of each of
// 16 rows of W.
constexpr int kTK = 128;
constexpr int kTN = 128;

template <class In, bool kAligned>
__device__ __attribute__((always_inline)) inline void quantize_cols_body(int64_t bx, int64_t by,
                                          const typename In::T* __restrict__ W, int64_t K,
                                          int64_t N, int64_t ldw,
                                          const uint32_t* __restrict__ colmax,
                                          uint8_t* __restrict__ Wq, int64_t ldq,
                                          float* __restrict__ sW) {
  __shared__ float inv_s[kTN];
  const int t = threadIdx.x;
  const int64_t n0 = bx * kTN;
  const int64_t k0 = by * kTK;
  if (t < kTN) {
    const int64_t n = n0 + t;
    float s = 0.0f, inv = 0.0f;
    if (n < N) {
      vector_scale(__uint_as_float(colmax[n]), s, inv);
      if (by == 0) sW[n] = s;
    }
    inv_s[t] = inv;
  }
  const int kg = t & 15, g = t >> 4;
  const int64_t c = n0 + g * 8;
  const int64_t valid = N - c;
  const int64_t kr = k0 + kg * 8;
  Vec8<In> v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (kr + u < K && valid > 0) {
      load8<In, kAligned>(W + (kr + u) * ldw + c, valid, v[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u].v[j] = typename In::T(0);
    }
  }
  __syncthreads();
  if (valid <= 0) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= valid) break;
    const float inv = inv_s[g * 8 + j];
    uint32_t word = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      // rows past K were loaded as zero and encode to the zero padding
      const uint32_t code =
          e2m1_magnitude(fabsf(In::widen(v[u].v[j])), inv) | (In::sign_bit(v[u].v[j]) << 3);
      word |= code << (4 * u);
    }
    *reinterpret_cast<uint32_t*>(Wq + (c + j) * ldq + kr / 2) = word;
  }
}

// Micro-scaled tile (bx, by): columns bx*128 .. +127, rows by*128 .. +127
// (rows past K read as zero and give the zero padding). Wave w takes block w, rows
// k0 + 32w .. +31: lane 4g + q owns rows 8q .. +7 of them in columns n0 + 8g .. +7,
// so that a load of the wave is 4 rows of 256 bytes (bfloat16), the 8 codes of one
// column are one 32-bit word and a quad of lanes shares a block. The words meet in
// LDS (a group of 8 columns every 528 bytes: the wave's 64 words lie in distinct
// banks) and leave as 16-byte pieces of whole columns, the scale bytes as words.
// Block scales go to the step-major array Ws (the
// byte of block b of column n at (b / 4) * 4ns + 4n + b % 4, ns the rows of that
// array: N, or those of all matrices whose scales share it). The 64 bytes of
// column n's codes in K step s go to Wq + n * ldq + s * step: with step 64 the
// codes of a column are one packed row of ldq bytes; with ldq 64 and step 64 N
// those of a step are together, and a tile's codes are 8 KiB in one piece.
// ldq and step are whole 64 bytes, Wq 16-byte and Ws 4-byte aligned. All threads
// of a workgroup of 256 call it. kNan: see BlockMax. (8 experts 4096 x 11008 with their product: 424 us; a
// wave over all four blocks of 32 columns, words stored as they come: 446. W with the
// non-temporal hint: 500, as the next call finds none of it in the last-level cache.)
constexpr int kMxTK = 128;  // codes along K per column tile
constexpr int kMxTN = 128;  // columns per tile

template <class In, bool kAligned, bool kNan = false>
__device__ __attribute__((always_inline)) inline void quantize_cols_mx_body(
    int64_t bx, int64_t by, const typename In::T* __restrict__ W, int64_t K, int64_t N,
    int64_t ldw, uint8_t* __restrict__ Wq, int64_t ldq, int64_t step, uint8_t* __restrict__ Ws,
    int64_t ns) {
  constexpr int kGroup = 8 * 64 + 16;  // bytes of 8 columns in LDS
  __shared__ __attribute__((aligned(16))) uint8_t codes[kMxTN / 8 * kGroup];
  __shared__ __attribute__((aligned(4))) uint8_t scales[kMxTN * 4];
  const int t = threadIdx.x;
  const int b = t >> 6, q = t & 3, g = (t >> 2) & 15;
  const int64_t n0 = bx * kMxTN;
  const int64_t c = n0 + g * 8;
  const int64_t valid = N - c;
  const int64_t kr = by * kMxTK + b * 32 + q * 8;
  Vec8<In> v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (kr + u < K && valid > 0) {
      load8<In, kAligned>(W + (kr + u) * ldw + c, valid, v[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u].v[j] = typename In::T(0);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    BlockMax<kNan> m;
#pragma unroll
    for (int u = 0; u < 8; ++u) m.take(fabsf(In::widen(v[u].v[j])));
    const int e = m.exponent();
    uint32_t word = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      word |= (mx_magnitude(fabsf(In::widen(v[u].v[j])), e) | (In::sign_bit(v[u].v[j]) << 3))
              << (4 * u);
    *reinterpret_cast<uint32_t*>(codes + g * kGroup + j * 64 + b * 16 + q * 4) = word;
    if (q == 0) scales[(g * 8 + j) * 4 + b] = uint8_t(e + 127);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = (i * 256 + t) * 16, col = at / 64;
    if (n0 + col < N)
      *reinterpret_cast<uint4*>(Wq + (n0 + col) * ldq + by * step + at % 64) =
          *reinterpret_cast<const uint4*>(codes + col / 8 * kGroup + at % 512);
  }
  if (t < kMxTN && n0 + t < N)
    *reinterpret_cast<uint32_t*>(Ws + by * 4 * ns + 4 * (n0 + t)) =
        *reinterpret_cast<const uint32_t*>(scales + t * 4);
}

// Row-wise (per row) micro-scaled quantization. Workgroup (bx, by) of gx x gy
// takes groups of kRows consecutive rows by, by + gy, ... and in each the chunks
// c = bx * 256 + t, c + 256 gx, ... (cpr = ldq / 4 chunks of 8 codes per padded
// row, a multiple of 16). Four consecutive t hold one block and sit on four
// consecutive lanes, and the chunk stride is a multiple of 4, so a block's lanes
// are active together. kRows rows are loaded before the first is encoded, so that
// a thread has that many loads in flight.
//
// Codes: rows in blocks of `block` rows (each block ldq bytes a row), and within a
// block the 64 bytes of every row's K step 0, then of step 1, ...: with block 1
// each row's codes are together (packed rows of ldq bytes), with block M those of
// a step. Scales are step-major over all M rows. |x| is clamped to tau, which makes
// tau of a NaN; kNan (see BlockMax): it is not.
template <class In, bool kFast, int kRows, bool kNan = false>
__device__ __attribute__((always_inline)) inline void quantize_rows_mx_body(
    int64_t bx, int64_t gx, int64_t by, int64_t gy, const typename In::T* __restrict__ X, int64_t M,
    int64_t K, int64_t ldx, float tau, uint8_t* __restrict__ Xq, int64_t ldq, int64_t block,
    uint8_t* __restrict__ Xs) {
  const int64_t cpr = ldq / 4;
  for (int64_t r0 = by * kRows; r0 < M; r0 += gy * kRows)
    for (int64_t c = bx * 256 + threadIdx.x; c < cpr; c += gx * 256) {
      Vec8<In> v[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        load_chunk<In, kFast>(X + (r0 + u < M ? r0 + u : M - 1) * ldx, c * 8, K, v[u]);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t r = r0 + u;
        if (r >= M) break;
        float ax[8];
        BlockMax<kNan> m;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ax[i] = fabsf(In::widen(v[u].v[i]));
          if constexpr (!kNan) ax[i] = fminf(ax[i], tau);
          m.take(ax[i]);
        }
        const int e = m.exponent();
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          word |= (mx_magnitude(ax[i], e) | (In::sign_bit(v[u].v[i]) << 3)) << (4 * i);
        const int64_t first = block == 1 ? r : r / block * block;
        *reinterpret_cast<uint32_t*>(Xq + first * ldq + (c / 16) * block * 64 + (r - first) * 64 +
                                     (c % 16) * 4) = word;
        // chunk c: block c / 4 = 4 * (c / 16) + (c / 4) % 4
        if ((c & 3) == 0) Xs[(c / 16) * 4 * M + 4 * r + ((c / 4) & 3)] = uint8_t(e + 127);
      }
    }
}

// Packed bytes from which a thread takes four rows (2048 x 5632 weights of 16
// experts: 97 us, one row a thread 123 us).
constexpr int64_t kManyRowBytes = int64_t(8) << 20;

// Workgroups: chunks of a row across x (at most 64), rows across y (at most 65535
// groups of `rows`).
inline dim3 mx_row_grid(int64_t M, int64_t cpr, int64_t rows) {
  const int64_t bx = (cpr + 255) / 256;
  const int64_t by = (M + rows - 1) / rows;
  return dim3(unsigned(bx < 64 ? bx : 64), unsigned(by < 65535 ? by : 65535));
}

}  // namespace fp4lin
