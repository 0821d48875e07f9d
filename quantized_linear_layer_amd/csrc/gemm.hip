// FP4 x FP4 GEMM on the gfx950 matrix cores with the scale epilogue.
//
// Role (FP4 training write-up "微软首创FP4训练框架", the GeMM-kernel paragraph): a
// dedicated FP4 matrix-multiply kernel stages packed FP4 tiles of A and B in
// shared memory, multiplies them block by block and reduces the partial
// results. That kernel simulated FP4 on FP8 tensor cores; here the product runs
// on CDNA4's native FP4 MFMA (v_mfma_scale_f32_32x32x64_f8f6f4 with both
// operands in E2M1 and unit E8M0 block scales, 127 = 2^0), accumulating in fp32.
// Every FP4 product is a multiple of 1/4 of magnitude <= 36 and |acc| <= 36*K,
// so the fp32 accumulation is exact for K < 2^24/144 whatever the order.
// (The 32x32x64 shape is used because on gfx950 it runs FP4 at twice the FP8
// rate; the 16x16x128 shape runs FP4 at the FP8 rate.)
//
// Epilogue (the granularity paragraph: row scales of A and column scales of W
// factor out of the K reduction, so they are applied once, after it):
//   Y[i,j] = RN32(RN32(acc[i,j] * sA[i]) * sB[j])
// With the sparse compensation matrix dA (the outlier and compensation
// paragraphs: dA = A - A_clamped, non-zero only where A was clamped, its
// product with the unquantized weight added back), the same epilogue adds
//   s[i,j] = sum over row i's non-zeros, k ascending, of val * W[k,j]
// (fp32 fused multiply-add from 0) to each element of a row that has
// non-zeros, before Y's only store: Y = Y0 + s. The result is bit-identical to
// the scaled product followed by the separate compensation kernel (spmm.hip),
// without reading Y back.
//
// Micro-scaled variant (kMx; the micro-scaling lecture "FP4量化训练的硬件挑战：
// NVIDIA Blackwell架构上的微缩放格式（Micro-scaling）实现", section 3, with the E8M0
// block scales of the format survey "训练大型语言模型的挑战"): A and B carry one
// E8M0 byte per 32 codes along K (mx.hip), which the instruction takes as its
// per-lane block-scale operands in place of the unit scales, and the epilogue
// writes the accumulator as it is: Y[i,j] = sum over blocks of
// 2^(eA + eB) * (block's FP4 dot product), accumulated in fp32.
//
// Layout and schedule:
//  * A is M x ldq bytes and B is N x ldq bytes, K-contiguous packed rows.
//  * A workgroup of 8 waves (4 x 2 grid, each wave 64 x 128 outputs) owns a
//    256 x 256 output tile and walks K in 128-code (64-byte) steps through
//    three LDS stages of 32 KiB. Operand tiles go from global memory straight
//    into LDS (buffer loads with an LDS destination, no register staging),
//    issued three steps ahead into the stage the previous step finished.
//    Each step issues its first 64-code sub-step of MFMAs, then waits for its
//    own loads of the next stage and meets the other waves at the barrier
//    while the matrix core works through the queued MFMAs, then issues the
//    next loads, the second sub-step of MFMAs and the next step's first
//    fragment reads. One workgroup per CU, two waves per SIMD. (Against
//    128 x 256 tiles with two 4-wave workgroups per CU, each wave moves 4
//    instead of 6 KiB of operands per step for the same 16 MFMAs: 3-13%
//    faster on the LLaMA shapes.)
//  * Each 16-byte chunk of a staged row is stored at a chunk index XOR-ed with
//    row bits, so that the lanes reading one chunk column of consecutive rows
//    hit distinct banks.
//  * For the 32x32x64 MFMA a lane supplies 32 consecutive codes (16 bytes) of
//    one row of A (lane % 32) and of one column of B (lane % 32); lanes 32..63
//    supply the next 32 codes. A and B use the same code-to-lane assignment,
//    so the k order inside the instruction does not matter for the exact sum.
//  * Tiles are visited in groups of 4 tile rows sweeping across N, and each of
//    the 8 XCDs (own L2 each; workgroups are dispatched round-robin over them)
//    takes a contiguous run of that order, so concurrent tiles on an XCD share
//    A rows and B columns in its L2.
//  * The scaled tile leaves through LDS: each wave writes two 32 x 32
//    fragments at a time into its own block of the (then idle) stage buffers
//    and stores them back as rows, 16 bytes per lane, so Y is written with
//    full-width stores of whole 256-byte row segments (4x fewer store
//    instructions than storing from the MFMA layout). The stores are
//    non-temporal: the output stream is not kept in L2 at the expense of the
//    operand tiles that concurrent workgroups re-read.
//  * With the compensation, the tile leaves in four chunks of 64 rows x all
//    256 columns (each wave row's 16 x 256 block in half a stage buffer).
//    After a barrier each wave finishes 8 whole rows of a chunk, one after the
//    other: a lane owns 4 consecutive columns, so a non-zero costs one 8-byte
//    (bf16 W) or 16-byte (fp32 W) gather per lane, addressed with the W row
//    offset in the scalar operand of a buffer load. A row's first 8 entries
//    (column, value) come in with one vector load by lanes 0..7 and reach the
//    wave through readlane; entries are loaded two rows ahead and gathered
//    one row ahead of the row being multiplied. Each row is stored once,
//    1 KiB per wave instruction.
#include <type_traits>

#include "device_common.hpp"
#include "gemm_core.hpp"
#include "internal.hpp"

namespace fp4lin {

namespace {

// Tiles of one launch: positions base .. base + nblocks / split - 1 of the
// order of a tiles_m x tiles_n grid, each cut into split tiles along M (split
// 2: the two 128-row halves of a 256-row tile).
struct TileMap {
  int base, tiles_m, tiles_n, split;
};

// Tile order: groups of G tile rows sweeping across N; each XCD takes a
// contiguous run of that order (a bijection from workgroup id to tile).
// kColumns: the tile columns one after another instead, each swept down M, so
// that the tiles an XCD runs together share one 256-column strip of the
// operands and of W (the compensation's gathers then stay in that XCD's L2).
template <bool kColumns = false>
__device__ inline void tile_coords(int bid, int nblocks, const TileMap& tmap, int& tm, int& tn) {
  const int xcd = bid & 7;
  const int idx = bid >> 3;
  const int base = nblocks >> 3, rem = nblocks & 7;
  const int t = xcd * base + (xcd < rem ? xcd : rem) + idx;
  if constexpr (kColumns) {
    tn = t / tmap.tiles_m;
    tm = t - tn * tmap.tiles_m;
    return;
  }
  const int u = tmap.base + t / tmap.split;  // position in the order
  const int half = t % tmap.split;
  const int tiles_m = tmap.tiles_m;
  constexpr int G = 4;
  const int per_group = G * tmap.tiles_n;
  const int grp = u / per_group;
  const int first_m = grp * G;
  const int gsize = (tiles_m - first_m) < G ? (tiles_m - first_m) : G;
  const int within = u - grp * per_group;
  tm = (first_m + within % gsize) * tmap.split + half;
  tn = within / gsize;
}

// The weight operand of the fused epilogue's compensation. The COO arrays
// are separate __restrict__ kernel arguments, which lets the compiler read a
// wave's entries with scalar loads (Y's stores cannot alias them).
struct CompArgs {
  const void* W;           // K x N weight, bf16 or fp32, row stride ldw elements
  int ldw;
  int w_bytes;             // K * ldw * element size (< 2^31)
  int w_vec;               // W rows allow 4-column vector loads
};

// One compensation gather: this lane's 4 columns of W row k (bf16: 8 bytes,
// fp32: 16 bytes), the row offset k * ldw in the scalar operand and the
// column offsets in vo (byte offsets of the lane's columns, each clamped into
// [0, N) so that every address lies inside row k whatever the lane: the
// buffer range check does not cover the scalar offset). With vector access
// (W and its row stride aligned to 4 elements and N a multiple of 4, so a
// lane's 4 columns are all below N or all past it, and lanes past N read the
// row's last 4) one load moves the 4 columns, vo[0] being their start;
// otherwise the 4 elements are loaded one by one.
template <bool kBf16W>
struct WSeg {
  uint32_t d[kBf16W ? 2 : 4];
};

template <bool kBf16W, bool kVec>
__device__ inline WSeg<kBf16W> load_wseg(__amdgpu_buffer_rsrc_t rs, const int (&vo)[4], int soff) {
  WSeg<kBf16W> w;
  if constexpr (kBf16W) {
    if constexpr (kVec) {
      const auto u = __builtin_amdgcn_raw_buffer_load_b64(rs, vo[0], soff, 0);
      w.d[0] = u[0];
      w.d[1] = u[1];
    } else {
      const uint32_t h0 = __builtin_amdgcn_raw_buffer_load_b16(rs, vo[0], soff, 0);
      const uint32_t h1 = __builtin_amdgcn_raw_buffer_load_b16(rs, vo[1], soff, 0);
      const uint32_t h2 = __builtin_amdgcn_raw_buffer_load_b16(rs, vo[2], soff, 0);
      const uint32_t h3 = __builtin_amdgcn_raw_buffer_load_b16(rs, vo[3], soff, 0);
      w.d[0] = h0 | (h1 << 16);
      w.d[1] = h2 | (h3 << 16);
    }
  } else {
    if constexpr (kVec) {
      const auto u = __builtin_amdgcn_raw_buffer_load_b128(rs, vo[0], soff, 0);
      w.d[0] = u[0];
      w.d[1] = u[1];
      w.d[2] = u[2];
      w.d[3] = u[3];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) w.d[c] = __builtin_amdgcn_raw_buffer_load_b32(rs, vo[c], soff, 0);
    }
  }
  return w;
}

// s[c] = fma(v, W[k, col + c], s[c]) for the lane's 4 columns.
template <bool kBf16W>
__device__ inline void fma_wseg(float v, const WSeg<kBf16W>& w, float (&s)[4]) {
  if constexpr (kBf16W) {
    s[0] = fmaf(v, __uint_as_float(w.d[0] << 16), s[0]);
    s[1] = fmaf(v, __uint_as_float(w.d[0] & 0xffff0000u), s[1]);
    s[2] = fmaf(v, __uint_as_float(w.d[1] << 16), s[2]);
    s[3] = fmaf(v, __uint_as_float(w.d[1] & 0xffff0000u), s[3]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] = fmaf(v, __uint_as_float(w.d[c]), s[c]);
  }
}

// Epilogue with the sparse compensation (see the header). The tile (BM x BN =
// 256 x 256, eight waves of 64 x 128 in a 4 x 2 grid) leaves in four chunks;
// chunk c holds the rows wm * 64 + (c >> 1) * 32 + (c & 1) * 16 + [0, 16) of
// all four wave rows wm, all 256 columns: wave row wm's 16 x 256 block is
// half (wm & 1) of stage wm >> 1 (with 128-row tiles of two wave rows, the
// whole of stage wm). Wave w then finishes the 8 rows
// (w & 1) * 8 + [0, 8) of wave row w >> 1's block. A block row is 256 floats
// (two blocks fill a stage); the 32-float halves of its 128-byte groups swap
// in rows with bit 2 set (lds_col), so that the lanes 32..63 of a staging
// write, four rows below lanes 0..31, hit the other 32 banks, while a row
// still reads back as 64 16-byte pieces.
template <class C, bool kMx, bool kBf16W, bool kWVec>
__device__ __attribute__((always_inline)) inline void fused_epilogue(
    v16f (&acc)[C::FM][C::FN], const float (&sa)[C::FM][16], const float (&sb)[C::FN],
    uint8_t* st0, uint8_t* st1, int wave, int wm, int wn, int lane, int m0, int n0, int M, int N,
    float* __restrict__ Y, int64_t ldy, const CompArgs& cp, const int32_t* __restrict__ row_ptr,
    const int32_t* __restrict__ col, const float* __restrict__ val) {
  constexpr int FM = C::FM, FN = C::FN, BN = C::BN;
  static_assert(C::BM == 64 * C::WM && (C::WM == 2 || C::WM == 4) && BN == 256 && C::WN == 2 &&
                    FM == 2 && FN == 4,
                "chunk layout of the fused epilogue");
  constexpr int kPitch = BN;  // floats
  constexpr int kPerStage = C::WM / 2;  // 16-row blocks per stage buffer (wave rows / 2 stages)
  static_assert(kPerStage * 16 * kPitch * 4 <= C::kStageBytes, "the blocks fit two stages");
  // LDS column of column c in block row r
  auto lds_col = [](int r, int c) { return c ^ (((r >> 2) & 1) << 5); };
  // non-zeros per gather group (one group per row is in flight ahead)
  constexpr int G = 8;

  // scales applied once, in place (the accumulators are then the output)
  if constexpr (!kMx) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          acc[fm][fn][r] = __fmul_rn(__fmul_rn(acc[fm][fn][r], sa[fm][r]), sb[fn]);
  }
  float* const wblk =
      reinterpret_cast<float*>(wm < kPerStage ? st0 : st1) + (wm % kPerStage) * 16 * kPitch;
  const int pr = wave >> 1, ph = wave & 1;
  const float* const rblk = reinterpret_cast<const float*>(pr < kPerStage ? st0 : st1) +
                            (pr % kPerStage) * 16 * kPitch + ph * 8 * kPitch;
  const int c4 = 4 * lane;
  const int gc = n0 + c4;
  constexpr int esz = kBf16W ? 2 : 4;
  const __amdgpu_buffer_rsrc_t rsW =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(cp.W), 0, cp.w_bytes, kBufferFlags);
  const int row_bytes = cp.ldw * esz;
  // byte offsets of this lane's 4 columns inside a W row, clamped below N
  // (vector access: the 4-column group itself, the last one for lanes past N)
  int voffW[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int cc = kWVec ? (gc + 4 <= N ? gc : N - 4) + c : (gc + c < N ? gc + c : N - 1);
    voffW[c] = cc * esz;
  }
  // the whole tile width lies below N and Y takes 16-byte stores (uniform)
  const bool y_full = ((reinterpret_cast<uintptr_t>(Y) & 15) == 0) && ((ldy & 3) == 0) &&
                      n0 + BN <= N;
  // Row boundaries come through the constant address space as scalar loads
  // (the COO is read-only while the kernel runs). The entries themselves
  // (column, value) are read as buffers that return zero at or past nnz, a
  // group of G by lanes 0 .. G-1 of one vector load, and reach the wave as
  // scalars through readlane: the scalar unit, which a CU shares among its
  // waves, is left almost nothing to do per non-zero (with scalar entry
  // loads, bounds clamps, per-slot weight masks and a search of the row
  // boundaries it ran about 30 scalar instructions per non-zero and set the
  // pace of the whole epilogue).
  typedef const __attribute__((address_space(4))) int32_t cint32;
  cint32* const rp_c = (cint32*)row_ptr;
  // nnz <= capacity <= 10 M (this schedule's limit) and M < 2^25 (packed rows
  // of at least 64 bytes addressed with 32-bit offsets), so byte offsets of
  // entries fit 32 bits
  const int nnz = rp_c[M];
  const __amdgpu_buffer_rsrc_t rsCol =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<int32_t*>(col), 0, nnz * 4, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsVal =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(val), 0, nnz * 4, kBufferFlags);
  // entries e0 .. e0+G-1: lane u < G gets entry e0 + u (zero past nnz)
  auto load_entries = [&](int e0, int& cv, float& vv) {
    const int voff = lane < G ? (e0 + lane) * 4 : nnz * 4;
    cv = __builtin_amdgcn_raw_buffer_load_b32(rsCol, voff, 0, 0);
    vv = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsVal, voff, 0, 0));
  };
  // the G gathers of a group whose first n entries are the row's (n may
  // exceed G): slots past n take weight 0 (0 * w adds nothing, so the fp32
  // sum keeps its value) and read the W row of whatever entry they hold
  auto gather = [&](int cv, float vv, int n, WSeg<kBf16W> (&w)[G], float (&wt)[G]) {
    const int offv = cv * row_bytes;  // < K * ldw * element size < 2^31
    const float vm = lane < n ? vv : 0.0f;
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int so = __builtin_amdgcn_readlane(offv, u);
      wt[u] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vm), u));
      w[u] = load_wseg<kBf16W, kWVec>(rsW, voffW, so);
    }
  };

  // Rows g0 .. g0+7 of the chunk just staged (their LDS rows at rblk, which
  // only this wave touches until the next barrier), one row after the other
  // in compile-time order. A row's first G non-zeros are one group; its
  // entries are loaded two rows ahead and its gathers one row ahead, so the
  // gathers of row j+1 are in flight while row j is multiplied. The rare
  // longer rows take their further groups one at a time after the first.
  // Every row, empty or not, issues the same loads, so the counter waits the
  // compiler places stay exact; then Y0 + s goes into the row's LDS row. No
  // store is issued in the loop: the 8 rows leave for Y after it.
  auto finish_rows = [&](int g0) {
    float* const rows = const_cast<float*>(rblk);
    // the 9 row boundaries (rows past M have no entries)
    int rp[9];
#pragma unroll
    for (int j = 0; j < 9; ++j) rp[j] = rp_c[g0 + j < M ? g0 + j : M];
    if (rp[0] < rp[8]) {
      int ce[2];
      float ve[2];
      WSeg<kBf16W> wq[2][G];
      float wt[2][G];
      load_entries(rp[0], ce[0], ve[0]);
      load_entries(rp[1], ce[1], ve[1]);
      gather(ce[0], ve[0], rp[1] - rp[0], wq[0], wt[0]);
      auto row = [&](auto j_c) {
        constexpr int j = decltype(j_c)::value;
        if constexpr (j + 2 <= 7) load_entries(rp[j + 2], ce[j & 1], ve[j & 1]);
        if constexpr (j + 1 <= 7)
          gather(ce[(j + 1) & 1], ve[(j + 1) & 1], rp[j + 2] - rp[j + 1], wq[(j + 1) & 1],
                 wt[(j + 1) & 1]);
        float acc4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < G; ++u) fma_wseg<kBf16W>(wt[j & 1][u], wq[j & 1][u], acc4);
        // further groups of a row of more than G non-zeros
        for (int e0 = rp[j] + G; e0 < rp[j + 1]; e0 += G) {
          int cv;
          float vv;
          load_entries(e0, cv, vv);
          WSeg<kBf16W> w[G];
          float t[G];
          gather(cv, vv, rp[j + 1] - e0, w, t);
#pragma unroll
          for (int u = 0; u < G; ++u) fma_wseg<kBf16W>(t[u], w[u], acc4);
        }
        if (rp[j + 1] > rp[j]) {
          float* const p = rows + j * kPitch + lds_col(j, c4);
          f32x4 y = *reinterpret_cast<const f32x4*>(p);
          y[0] = __fadd_rn(y[0], acc4[0]);
          y[1] = __fadd_rn(y[1], acc4[1]);
          y[2] = __fadd_rn(y[2], acc4[2]);
          y[3] = __fadd_rn(y[3], acc4[3]);
          *reinterpret_cast<f32x4*>(p) = y;
        }
      };
      row(std::integral_constant<int, 0>{});
      row(std::integral_constant<int, 1>{});
      row(std::integral_constant<int, 2>{});
      row(std::integral_constant<int, 3>{});
      row(std::integral_constant<int, 4>{});
      row(std::integral_constant<int, 5>{});
      row(std::integral_constant<int, 6>{});
      row(std::integral_constant<int, 7>{});
    }
    // the 8 rows, Y0 + s (rows without non-zeros: Y0 as it is), to Y
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int gr = g0 + i;
      const f32x4 y = *reinterpret_cast<const f32x4*>(rows + i * kPitch + lds_col(i, c4));
      if (gr < M) {
        float* dst = Y + int64_t(gr) * ldy + gc;
        if (y_full) {
          __builtin_nontemporal_store(y, reinterpret_cast<f32x4*>(dst));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (gc + c < N) dst[c] = y[c];
        }
      }
    }
  };

  // acc element r of fragment row fm holds row 8 * (r >> 2) + 4 * (lane >> 5)
  // + (r & 3) of the fragment: elements h * 8 .. h * 8 + 7 are its rows
  // h * 16 + [0, 16)
  auto stage_chunk = [&](auto fm_c, auto h_c) {
    constexpr int fm = decltype(fm_c)::value, h = decltype(h_c)::value;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int rr = 0; rr < 8; ++rr) {
        const int rl = 8 * (rr >> 2) + 4 * (lane >> 5) + (rr & 3);
        wblk[rl * kPitch + lds_col(rl, wn * (FN * 32) + fn * 32 + (lane & 31))] =
            acc[fm][fn][h * 8 + rr];
      }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
#pragma nounroll
  for (int c = 0; c < 4; ++c) {
    switch (c) {
      case 0: stage_chunk(I0{}, I0{}); break;
      case 1: stage_chunk(I0{}, I1{}); break;
      case 2: stage_chunk(I1{}, I0{}); break;
      default: stage_chunk(I1{}, I1{}); break;
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(63, 0));
    raw_barrier();
    finish_rows(m0 + pr * 64 + (c >> 1) * 32 + (c & 1) * 16 + ph * 8);
    // every wave's LDS reads of this chunk are done before the next is staged
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(63, 0));
    raw_barrier();
  }
}

// Tile order of the kernels with the fused compensation (see tile_coords).
constexpr bool kFusedColumns = true;

// Largest COO capacity per row of A for which the compensation runs in the
// GEMM's epilogue (see run_gemm).
constexpr int64_t kFusedMaxPerRow = 10;

// kComp: 0 no compensation; with it, 1 + (W is float32) + 2 * (W rows allow
// 4-column vector gathers): 1 / 3 bfloat16 W, 2 / 4 float32 W.
template <class C, bool kMx, int kComp>
__global__ __launch_bounds__(C::kThreads, C::kMinBlocks) void fp4_gemm_kernel(
    const uint8_t* __restrict__ Aq, const float* __restrict__ sA,
    const uint8_t* __restrict__ Bq, const float* __restrict__ sB, int M, int N, int ldq,
    TileMap tmap, float* __restrict__ Y, int64_t ldy, const uint8_t* __restrict__ As,
    const uint8_t* __restrict__ Bs, CompArgs cp, const int32_t* __restrict__ row_ptr,
    const int32_t* __restrict__ col, const float* __restrict__ val) {
  constexpr int BM = C::BM, BN = C::BN, WN = C::WN, BKB = C::BKB;
  constexpr int FM = C::FM, FN = C::FN;
  constexpr int SB = C::kStageBytes;
  // Three LDS stages, separate objects so that the compiler can tell the
  // direct-to-LDS loads into one stage from the fragment reads of another.
  __shared__ __attribute__((aligned(16))) uint8_t st0[SB];
  __shared__ __attribute__((aligned(16))) uint8_t st1[SB];
  __shared__ __attribute__((aligned(16))) uint8_t st2[SB];

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN;
  const int wn = wave % WN;
  int tm, tn;
  tile_coords<(kComp != 0) && kFusedColumns>(blockIdx.x, gridDim.x, tmap, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int nkt = (ldq + BKB - 1) / BKB;

  using Feed = Fp4Feed<C, kMx>;
  const int nblk = ldq / 16;
  Feed f(Fp4Operand{Aq, ldq, BKB, M, M * ldq, As, 4 * M, M * nblk},
         Fp4Operand{Bq, ldq, BKB, N, N * ldq, Bs, 4 * N, N * nblk}, m0, n0, wave, lane);
  gemm_pipeline(f, nkt, st0, st1, st2);
  auto& acc = f.acc;

  // ---- epilogue -------------------------------------------------------------
  // Scales are applied in the MFMA output layout: for accumulator element r,
  // lanes 0..31 hold 32 consecutive columns of one row and lanes 32..63 the
  // same columns four rows down. All row and column scales of the lane are
  // loaded before any is used.
  // (With block scales the accumulator is the output and no scale is loaded.)
  const int col_l = lane & 31;
  float sb[FN];
  float sa[FM][16];
  if constexpr (!kMx) {
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
      const int gc = n0 + wn * (FN * 32) + fn * 32 + col_l;
      sb[fn] = (gc < N) ? sB[gc] : 0.0f;
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int gr = m0 + wm * (FM * 32) + fm * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        sa[fm][r] = (gr < M) ? sA[gr] : 0.0f;
      }
  }
  if constexpr (kComp != 0) {
    fused_epilogue<C, kMx, (kComp & 1) != 0, kComp >= 3>(acc, sa, sb, st0, st1, wave, wm, wn,
                                                          lane, m0, n0, M, N, Y, ldy, cp,
                                                          row_ptr, col, val);
    return;
  }
  store_tile<C>(st0, st1, st2, wave, lane, m0, n0, M, N, Y, ldy, [&](int fm, int fn, int r) {
    return kMx ? acc[fm][fn][r] : __fmul_rn(__fmul_rn(acc[fm][fn][r], sa[fm][r]), sb[fn]);
  });
}

// Tiles of the GEMM without compensation: 256 x 256 (eight waves, one
// workgroup per CU) once the grid fills the 256 CUs twice, 128 x 256 (four
// waves, two workgroups per CU) below that, where finer tiles balance better
// (LLaMA 1.3B up, 352 large tiles: 45.6 against 41.6 us).
using GemmTile = GemmCfg<256, 256, 4, 2, 64, 1>;
using GemmSmallTile = GemmCfg<128, 256, 2, 2, 64, 2>;
constexpr int kLargeTilesMin = 512;
constexpr int kCUs = 256;  // MI355X
// Tile of the GEMM with the compensation in its epilogue: the two workgroups
// on a CU keep the matrix core busy in turn while either one gathers (13B up:
// 509 against 521 us with 256 x 256 tiles).
using GemmFusedTile = GemmCfg<128, 256, 2, 2, 64, 2>;

// The GEMM without compensation over positions base .. base + count - 1 of
// the order of a tiles_m x tiles_n grid of 256 x 256 tiles (C: those tiles,
// or with 128-row C their two halves).
template <class C, bool kMx>
hipError_t launch_plain(const uint8_t* Aq, const float* sA, const uint8_t* Bq, const float* sB,
                        const uint8_t* As, const uint8_t* Bs, int64_t M, int64_t N, int64_t ldq,
                        float* Y, int64_t ldy, const TileMap& tmap, int count,
                        hipStream_t stream) {
  fp4_gemm_kernel<C, kMx, 0><<<dim3(unsigned(count * tmap.split)), C::kThreads, 0, stream>>>(
      Aq, sA, Bq, sB, int(M), int(N), int(ldq), tmap, Y, ldy, As, Bs, CompArgs{nullptr, 0, 0, 0},
      nullptr, nullptr, nullptr);
  return hipGetLastError();
}

template <bool kMx>
hipError_t run_gemm(const uint8_t* Aq, const float* sA, const uint8_t* Bq, const float* sB,
                    const uint8_t* As, const uint8_t* Bs, int64_t M, int64_t N, int64_t ldq,
                    const SparseArgs& sp, float* Y, int64_t ldy, hipStream_t stream) {
  // K steps are whole 64-byte chunks of the packed rows (the packed row length
  // is a multiple of 64 bytes), so no step reads past a row.
  static_assert(GemmTile::BKB == 64 && GemmSmallTile::BKB == 64 && GemmFusedTile::BKB == 64,
                "one K step per 64 bytes");
  if (ldq % 64 != 0) return hipErrorInvalidValue;
  // The two schedules of the compensation give the same bits. The fused
  // epilogue saves the read-modify-write of Y (8 bytes per output), but its
  // gathers run in the GEMM's waves (two per SIMD), which hide memory latency
  // worse than the separate kernel's eight, and it needs the 128 x 256 tile.
  // Measured on the LLaMA-shaped workloads (GEMM with compensation, us,
  // fused against the large-tile GEMM + separate kernel): 13B up 5.1/row
  // 437-459 against 295 + 215; 13B down 13.8/row 384 against 364; 1.3B up
  // 20/row 144 against 112; 7B up 41/row 948 against 656. The COO's capacity
  // bounds the non-zeros (for the select's own COO it is M*K*(1-q)).
  const bool fused = sp.row_ptr != nullptr && sp.capacity <= kFusedMaxPerRow * M;
  if (!fused) {
    static_assert(GemmTile::BM == 2 * GemmSmallTile::BM && GemmTile::BN == GemmSmallTile::BN,
                  "a large tile is two small ones");
    const int tiles_m = int((M + GemmTile::BM - 1) / GemmTile::BM);
    const int tiles_n = int((N + GemmTile::BN - 1) / GemmTile::BN);
    const int large = tiles_m * tiles_n;
    hipError_t e;
    if (large >= kLargeTilesMin) {
      // whole rounds of large tiles (one per CU), then, when at most half a
      // round is left, the rest of the order as 128-row halves, two
      // workgroups per CU: a last round of large tiles would leave most CUs
      // idle (7B, 96 left: 231 against 222 us; 13B down, 128 left: 279
      // against 264), while a fuller one runs better as large tiles (13B up,
      // 192 left: 293 against 300)
      const int rest = large % kCUs;
      const int whole = rest <= kCUs / 2 ? large - rest : large;
      e = launch_plain<GemmTile, kMx>(Aq, sA, Bq, sB, As, Bs, M, N, ldq, Y, ldy,
                                      TileMap{0, tiles_m, tiles_n, 1}, whole, stream);
      if (e == hipSuccess && whole < large)
        e = launch_plain<GemmSmallTile, kMx>(Aq, sA, Bq, sB, As, Bs, M, N, ldq, Y, ldy,
                                             TileMap{whole, tiles_m, tiles_n, 2}, large - whole,
                                             stream);
    } else {
      e = launch_plain<GemmSmallTile, kMx>(Aq, sA, Bq, sB, As, Bs, M, N, ldq, Y, ldy,
                                           TileMap{0, tiles_m, tiles_n, 2}, large, stream);
    }
    if (e != hipSuccess || sp.row_ptr == nullptr) return e;
    return launch_sparse_add(sp, M, N, Y, ldy, stream);
  }
  CompArgs cp{nullptr, 0, 0, 0};
  using CF = GemmFusedTile;
  const int tiles_mf = int((M + CF::BM - 1) / CF::BM);
  const int tiles_nf = int((N + CF::BN - 1) / CF::BN);
  const int64_t esz = sp.w_bf16 ? 2 : 4;
  // 4-column vector gathers need every W row start aligned to 4 elements
  // (8 bytes for bf16, 16 for fp32) and N a multiple of 4 (no lane straddles N)
  const bool w_vec = (reinterpret_cast<uintptr_t>(sp.W) % (4 * esz) == 0) && (sp.ldw % 4 == 0) &&
                     (N % 4 == 0);
  cp = CompArgs{sp.W, int(sp.ldw), int(sp.w_rows * sp.ldw * esz), w_vec ? 1 : 0};
  const int mode = (sp.w_bf16 ? 1 : 2) + (w_vec ? 2 : 0);
#define FP4LIN_GEMM_COMP(MODE)                                                                  \
  case MODE:                                                                                    \
    fp4_gemm_kernel<CF, kMx, MODE><<<dim3(unsigned(tiles_mf * tiles_nf)), CF::kThreads, 0,      \
                                     stream>>>(                                                 \
        Aq, sA, Bq, sB, int(M), int(N), int(ldq), TileMap{0, tiles_mf, tiles_nf, 1}, Y, ldy, As, \
        Bs, cp, sp.row_ptr,                                                                     \
        sp.col, sp.val);                                                                        \
    break;
  switch (mode) {
    FP4LIN_GEMM_COMP(1)
    FP4LIN_GEMM_COMP(2)
    FP4LIN_GEMM_COMP(3)
    FP4LIN_GEMM_COMP(4)
    default: return hipErrorInvalidValue;
  }
#undef FP4LIN_GEMM_COMP
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_gemm(const uint8_t* Aq, const float* sA, const uint8_t* Bq, const float* sB,
                           int64_t M, int64_t N, int64_t ldq, const SparseArgs& sp, float* Y,
                           int64_t ldy, hipStream_t stream) {
  return run_gemm<false>(Aq, sA, Bq, sB, nullptr, nullptr, M, N, ldq, sp, Y, ldy, stream);
}

hipError_t launch_fp4_gemm_mx(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                              const uint8_t* Bs, int64_t M, int64_t N, int64_t ldq,
                              const SparseArgs& sp, float* Y, int64_t ldy, hipStream_t stream) {
  return run_gemm<true>(Aq, nullptr, Bq, nullptr, As, Bs, M, N, ldq, sp, Y, ldy, stream);
}

}  // namespace fp4lin
