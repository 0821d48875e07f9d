// Operand feed of the unquantized products (bfloat16 or float32 operands, fp32
// accumulation) for the GEMM pipeline of gemm_core.hpp: K steps of 64 bytes a
// row, 32 bfloat16 or 16 float elements.
//
// An operand is a matrix of `extent` output rows (or columns) by `k` elements of
// the reduction, in memory either along the reduction (kT false: element (i, j)
// at p[i * ld + j]) or across it (kT true: at p[j * ld + i]). Both are staged by
// 16-byte loads straight into LDS and read back as MFMA fragments, so no matrix
// is ever transposed in memory:
//  * along: 64-byte rows, as the FP4 feed stages them; a lane's 16 bytes of a
//    fragment are consecutive in the reduction.
//  * across: rows of the reduction, BM elements each. bfloat16 fragments come
//    out of the transposing LDS read: 16 lanes name 4 reduction rows x 16
//    columns (8 bytes each) and lane i gets column i's four values. float32
//    fragments are read element by element, 32 consecutive columns a half wave.
//    64-byte (bfloat16) or 128-byte (float32) segments of a staged row are
//    XOR-swizzled with the reduction row, so that the rows one read touches
//    lie in distinct banks.
// For the 32x32 shapes a lane supplies the row (lane % 32) and one half of the
// reduction range of a sub-step (lane / 32); A and B use the same assignment, so
// the order inside a sub-step does not matter. A 16-byte fragment holds the
// operand of one 32x32x16 bfloat16 MFMA or of four 32x32x2 float32 ones.
//
// Requirements, checked by the callers: p 16-byte aligned, ld * size a multiple
// of 16, and the contiguous size (k along, extent across) a multiple of 8
// elements, so that every 16-byte piece lies wholly inside a row or outside.
// Pieces past either size read as zero.
#pragma once

#include "gemm_core.hpp"

namespace fp4lin {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <class T>
struct DenseOperand {
  const T* p;
  int64_t ld;
  int extent, k;
};

template <class T>
constexpr int kStepElems = 64 / int(sizeof(T));  // reduction elements of a K step

template <class C, class T, bool kAT, bool kBT>
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
    A.p += kAT ? m0 : m0 * A.ld;
    A.extent -= m0;
    B.p += kBT ? n0 : n0 * B.ld;
    B.extent -= n0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool is_a = j < kPerA;
      const int b = wave + (is_a ? j : j - kPerA) * kWaves;  // block of the operand
      src_off[j] = is_a ? offset<BM, kAT>(A, b) : offset<BN, kBT>(B, b);
    }
  }

  // Source byte offset (from the operand's tile, its first K step) of this
  // lane's 16 bytes of 1 KiB block b; past the extent: outside any resource.
  template <int BX, bool kT>
  __device__ inline int offset(const DenseOperand<T>& o, int b) const {
    if constexpr (kT) {
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

  template <int BX, bool kT, int J0, int J1>
  __device__ inline void load(const DenseOperand<T>& o, int kt, uint8_t* dst) {
    const int k0 = kt * kE;
    if constexpr (kT) {
      // the resource starts at the step's first reduction row and ends with its
      // last one inside k, so rows past k read as zero (and a step past k has none:
      // (left - 1) * ld + cols <= 0 there, as ld >= cols)
      const int left = o.k - k0 < kE ? o.k - k0 : kE;
      const int cols = o.extent < BX ? o.extent : BX;
      const int ldb = int(o.ld * int64_t(sizeof(T)));
      const int end = (left - 1) * ldb + cols * int(sizeof(T));
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<T*>(o.p + int64_t(k0) * o.ld), 0, end > 0 ? end : 0, kBufferFlags);
#pragma unroll
      for (int j = J0; j < J1; ++j) load_lds16(rs, dst + (j - J0) * kWaves * 1024, src_off[j]);
    } else {
      const int rows = o.extent < BX ? o.extent : BX;
      const int bytes = int(((rows - 1) * o.ld + o.k) * int64_t(sizeof(T)));
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(o.p), 0, bytes, kBufferFlags);
      // this lane's piece of the step (the same of every block) lies inside k
      const int c = (lane & 3) ^ swz<CPR>(lane >> 2, 0);
      const bool in = k0 * int(sizeof(T)) + c * 16 < o.k * int(sizeof(T));
#pragma unroll
      for (int j = J0; j < J1; ++j)
        load_lds16(rs, dst + (j - J0) * kWaves * 1024,
                   in && src_off[j] != kOut ? src_off[j] + k0 * int(sizeof(T)) : kOut);
    }
  }

  __device__ inline void dma(int kt, uint8_t* stage) {
    load<BM, kAT, 0, kPerA>(A, kt, stage + wave * 1024);
    load<BN, kBT, kPerA, kPer>(B, kt, stage + BM * 64 + wave * 1024);
  }

  // Fragment of rows x0 .. x0 + 31 in the sub-step kk of the operand staged at
  // byte `at` of the stage. (Every address is one offset from the stage's own
  // array: through longer chains the compiler loses which array a read is from
  // and waits for all loads in flight.)
  template <int BX, bool kT>
  __device__ inline Frag frag(const uint8_t* stage, int at, int x0, int kk) const {
    if constexpr (!kT) {
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
