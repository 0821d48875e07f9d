// Operand feed of the unquantized products (bfloat16 or float32 operands, fp32
// accumulation) for the GEMM pipeline of gemm_core.hpp: K steps of 64 bytes a
// row, 32 bfloat16 or 16 float elements.
//
// An operand is a matrix of `extent` output rows (or columns) by `k` elements of
// the reduction, in one of three orders:
//  * kAlong: element (i, j) at p[i * ld + (j / kE) * step + j % kE], kE the
//    elements of a K step: rows along the reduction (step kE), or the rows of a
//    step together (ld kE, step kE times the rows). The second makes a tile's
//    step whole cache lines, where 64 bytes of a longer row are half of one and
//    twice the requests to L2.
//  * kAcross: element (i, j) at p[j * ld + i]: rows across the reduction.
//  * kPieces (bfloat16): element (i, j) at p[(i / 32) * step + j * 32 + i % 32]:
//    the second form of kAlong of a matrix whose rows are this operand's
//    reduction.
// All are staged by 16-byte loads straight into LDS and read back as MFMA
// fragments, so no matrix is ever transposed in memory:
//  * along: rows of a step's bytes, as the FP4 feed stages them; a lane's 16
//    bytes of a fragment are consecutive in the reduction.
//  * across: rows of the reduction, BM elements each. bfloat16 fragments come
//    out of the transposing LDS read: 16 lanes name 4 reduction rows x 16
//    columns (8 bytes each) and lane i gets column i's four values. float32
//    fragments are read element by element, 32 consecutive columns a half wave.
//    64-byte (bfloat16) or 128-byte (float32) segments of a staged row are
//    XOR-swizzled with the reduction row, so that the rows one read touches
//    lie in distinct banks.
//  * pieces: the step's 32 reduction rows of one 32-column piece after the other,
//    64 bytes each: the four rows of a transposing read are 256 bytes in a row.
// For the 32x32 shapes a lane supplies the row (lane % 32) and one half of the
// reduction range of a sub-step (lane / 32); A and B use the same assignment, so
// the order inside a sub-step does not matter. A 16-byte fragment holds the
// operand of one 32x32x16 bfloat16 MFMA or of four 32x32x2 float32 ones.
//
// Requirements, checked by the callers: p 16-byte aligned, ld and step whole
// 16-byte pieces, and the contiguous size (k along, extent across) a multiple of 8
// elements, so that every 16-byte piece lies wholly inside a row or outside.
// Pieces past either size read as zero (kPieces: the rest of the last 32 columns
// is read as it is).
#pragma once

#include "gemm_core.hpp"

namespace fp4lin {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum { kAlong = 0, kAcross = 1, kPieces = 2 };

template <class T>
struct DenseOperand {
  const T* p;
  int64_t ld, step;
  int extent, k;
};

template <class T>
constexpr int kStepElems = 64 / int(sizeof(T));  // reduction elements of a K step

template <class C, class T, int kAT, int kBT>
struct DenseFeed {
  static constexpr int BM = C::BM, BN = C::BN, WN = C::WN, CPR = C::CPR;
  static constexpr int FM = C::FM, FN = C::FN;
  static constexpr int kWaves = C::kThreads / kWave;
  static constexpr int kBlocks = C::kStageBytes / 1024;
  static constexpr int kPer = kBlocks / kWaves, kPerA = BM / 16 / kWaves;
  static_assert(C::BKB == 64 && C::kSub == 2, "64-byte K steps");
  static_assert(kBlocks % kWaves == 0 && (BM / 16) % kWaves == 0, "even block split");
  static constexpr int NS = 0, NL = 0;
  static constexpr int kE = kStepElems<T>;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kSegChunks = kBf16 ? 4 : 8;  // 16-byte pieces of a swizzled segment
  using Frag = s16x8;  // 16 bytes: 8 bfloat16 or 4 float

  v16f acc[FM][FN];
  DenseOperand<T> A, B;
  int src_off[kPer];
  int wave, lane;

  // swizzle key of a staged reduction row: the rows one fragment read touches
  // differ in it (bfloat16: 4 consecutive rows; float32: rows 4 apart)
  __device__ static inline int key(int row) { return kBf16 ? row & 3 : (row >> 2) & 1; }

  // byte offset, in a staged operand whose rows are BX elements of the output,
  // of element x of reduction row `row`
  template <int BX>
  __device__ static inline int across(int row, int x) {
    constexpr int kSeg = kSegChunks * 16 / int(sizeof(T));  // elements of a segment
    return row * (BX * int(sizeof(T))) + (((x / kSeg) ^ key(row)) * kSegChunks * 16) +
           (x % kSeg) * int(sizeof(T));
  }

  // the tile's first rows of the two operands are m0 and n0
  __device__ inline DenseFeed(const DenseOperand<T>& A_, const DenseOperand<T>& B_, int m0, int n0,
                              int wave_, int lane_)
      : A(A_), B(B_), wave(wave_), lane(lane_) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v16f{};
    // from here on the operands start at the tile
    A.p += at_row<kAT>(A, m0);
    A.extent -= m0;
    B.p += at_row<kBT>(B, n0);
    B.extent -= n0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool is_a = j < kPerA;
      const int b = wave + (is_a ? j : j - kPerA) * kWaves;  // block of the operand
      src_off[j] = is_a ? offset<BM, kAT>(A, b) : offset<BN, kBT>(B, b);
    }
  }

  // Elements from row 0 to row x (of the output; a tile's, so a multiple of 32).
  template <int kT>
  __device__ static inline int64_t at_row(const DenseOperand<T>& o, int x) {
    return kT == kAlong ? x * o.ld : kT == kAcross ? int64_t(x) : x / 32 * o.step;
  }

  // Source byte offset (from the operand's tile and its K step) of this lane's
  // 16 bytes of 1 KiB block b; past the extent: outside any resource.
  template <int BX, int kT>
  __device__ inline int offset(const DenseOperand<T>& o, int b) const {
    if constexpr (kT == kPieces) {
      // block b: 16 reduction rows of piece b / 2
      return (b >> 1) * 32 < o.extent
                 ? int((b >> 1) * o.step * int64_t(sizeof(T))) + (b & 1) * 1024 + lane * 16
                 : kOut;
    } else if constexpr (kT == kAcross) {
      constexpr int kChunks = BX * int(sizeof(T)) / 16;  // of a staged row
      const int row = b * (64 / kChunks) + lane / kChunks;
      const int at = lane % kChunks;  // physical piece
      const int c = (((at / kSegChunks) ^ key(row)) * kSegChunks) + at % kSegChunks;
      const int x = c * 16 / int(sizeof(T));
      return x < o.extent ? int(row * o.ld * int64_t(sizeof(T))) + c * 16 : kOut;
    } else {
      const int r = b * 16 + (lane >> 2);
      const int c = (lane & 3) ^ swz<CPR>(r, 0);
      return r < o.extent ? int(r * o.ld * int64_t(sizeof(T))) + c * 16 : kOut;
    }
  }
  static constexpr int kOut = 0x7fffffff;

  // Loads J0 .. J1 - 1 (blocks of one operand) of step kt. The resource starts at
  // the step and ends with what of it lies inside k; a step past k has none.
  template <int BX, int kT, int J0, int J1>
  __device__ inline void load(const DenseOperand<T>& o, int kt, uint8_t* dst) {
    const int left = o.k - kt * kE < kE ? o.k - kt * kE : kE;  // of the reduction
    const int most = o.extent < BX ? o.extent : BX;            // of the output
    const int ldb = int(o.ld * int64_t(sizeof(T)));
    const T* p;
    int bytes;
    bool in = true;  // this lane's pieces (the same of every block) lie inside k
    if constexpr (kT == kAlong) {
      p = o.p + kt * o.step;
      bytes = (most - 1) * ldb + left * int(sizeof(T));
      in = ((lane & 3) ^ swz<CPR>(lane >> 2, 0)) * 16 < left * int(sizeof(T));
    } else if constexpr (kT == kAcross) {
      // (left - 1) * ld + most <= 0 where left <= 0, as ld >= most
      p = o.p + kt * kE * o.ld;
      bytes = (left - 1) * ldb + most * int(sizeof(T));
    } else {
      p = o.p + int64_t(kt) * kE * 32;
      bytes = (most - 1) / 32 * int(o.step * int64_t(sizeof(T))) + left * 64;
      in = (wave & 1) * 16 + (lane >> 2) < left;  // kWaves is even: every block's rows
      static_assert(kT != kPieces || kWaves % 2 == 0, "");
    }
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<T*>(p), 0, left > 0 && bytes > 0 ? bytes : 0, kBufferFlags);
#pragma unroll
    for (int j = J0; j < J1; ++j)
      load_lds16(rs, dst + (j - J0) * kWaves * 1024, in ? src_off[j] : kOut);
  }

  __device__ inline void dma(int kt, uint8_t* stage) {
    load<BM, kAT, 0, kPerA>(A, kt, stage + wave * 1024);
    load<BN, kBT, kPerA, kPer>(B, kt, stage + BM * 64 + wave * 1024);
  }

  // Fragment of rows x0 .. x0 + 31 in the sub-step kk of the operand staged at
  // byte `at` of the stage. (Every address is one offset from the stage's own
  // array: through longer chains the compiler loses which array a read is from
  // and waits for all loads in flight.)
  template <int BX, int kT>
  __device__ inline Frag frag(const uint8_t* stage, int at, int x0, int kk) const {
    if constexpr (kT == kPieces) {
      const int g = lane >> 4, i = lane & 15;
      const int row = kk * 16 + 8 * (g >> 1) + (i >> 2);
      const int p = at + x0 * 64 + row * 64 + (16 * (g & 1) + (i & 3) * 4) * 2;
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(stage + p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(stage + (p + 4 * 64)));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else if constexpr (kT == kAlong) {
      const int r = x0 + (lane & 31);
      const int c = kk * 2 + (lane >> 5);
      return *reinterpret_cast<const Frag*>(stage + (at + r * 64 + (swz<CPR>(r, c) << 4)));
    } else if constexpr (kBf16) {
      const int g = lane >> 4, i = lane & 15;
      const int row = kk * 16 + 8 * (g >> 1) + (i >> 2);
      const int x = x0 + 16 * (g & 1) + (i & 3) * 4;
      // rows row and row + 4 have the same swizzle key
      const int p = at + across<BX>(row, x);
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(stage + p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(stage + (p + 4 * BX * 2)));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      const int row = kk * 8 + 4 * (lane >> 5);
      const int p = at + across<BX>(row, x0 + (lane & 31));
      f32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float*>(stage + (p + j * BX * 4));
      return __builtin_bit_cast(Frag, v);
    }
  }

  __device__ inline void read_frags(const uint8_t* stage, int kk, Frag* af, Frag* bf) {
    const int wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) af[fm] = frag<BM, kAT>(stage, 0, (wm * FM + fm) * 32, kk);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
      bf[fn] = frag<BN, kBT>(stage, BM * 64, (wn * FN + fn) * 32, kk);
  }

  __device__ inline void load_scales(int, uint32_t*) {}
  __device__ inline void expand(const uint32_t*, uint32_t*) {}

  template <int KK>
  __device__ inline void mfmas(const Frag* af, const Frag* bf, const uint32_t*) {
    if constexpr (kBf16) {
#pragma unroll
      for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
          acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, af[fm]), __builtin_bit_cast(bf16x8, bf[fn]), acc[fm][fn],
              0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
          for (int fn = 0; fn < FN; ++fn)
            acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                __builtin_bit_cast(f32x4, af[fm])[j], __builtin_bit_cast(f32x4, bf[fn])[j],
                acc[fm][fn], 0, 0, 0);
    }
  }
};

}  // namespace fp4lin
