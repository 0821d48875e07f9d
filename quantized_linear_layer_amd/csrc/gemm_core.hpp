// The pieces that the GEMM kernels share: tile configurations, the LDS swizzle,
// direct-to-LDS loads, the three-stage K pipeline, the FP4 operand feed and the
// store of a finished tile. gemm.hip describes the schedule as a whole.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace fp4lin {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Word 3 of a raw buffer resource on gfx9-family parts (32-bit data format,
// no swizzle); with stride 0 the bounds check is offset < num_records.
constexpr int kBufferFlags = 0x00020000;

template <int BM_, int BN_, int WM_, int WN_, int BKB_, int MINB_>
struct GemmCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BKB = BKB_;
  static constexpr int kMinBlocks = MINB_;  // workgroups per CU the register budget targets
  static constexpr int kThreads = WM * WN * 64;
  static constexpr int FM = BM / WM / 32;
  static constexpr int FN = BN / WN / 32;
  static constexpr int CPR = BKB / 16;            // 16-byte chunks per staged row
  static constexpr int kSub = BKB / 32;            // 64-code MFMA steps per K step
  static constexpr int kStageBytes = (BM + BN) * BKB;
  static_assert(FM >= 1 && FN >= 1, "tile too small for the wave grid");
  static_assert(CPR == 4 || CPR == 8, "swizzle assumes 64- or 128-byte staged rows");
};

// s_waitcnt immediate of gfx9-family parts: vmcnt in bits 3:0 (and 15:14),
// expcnt in 6:4 (7: do not wait), lgkmcnt in 11:8.
constexpr int waitcnt_vm_lgkm(int vm, int lgkm) {
  return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8);
}

// The same with lgkmcnt left alone.
constexpr int waitcnt_vm(int vm) { return waitcnt_vm_lgkm(vm, 15); }

// Physical 16-byte chunk of logical chunk c in staged row r. A fragment read
// is a 128-bit LDS read of 32 consecutive rows at one logical chunk (lanes
// 32..63 at the next chunk). On gfx950 such a read takes 4 LDS cycles when
// every 16 consecutive lanes cover 64 distinct 4-byte banks, the rate of a
// contiguous 1 KiB read; measured on the device, the mapping below reaches
// it for 64-byte rows, while an unswizzled layout takes 16 cycles:
//   64-byte rows:  chunk ^ ((r >> 2) & 3)
//   128-byte rows: chunk ^ ((r ^ (r >> 3)) & 7)
template <int CPR>
__device__ inline int swz(int r, int c) {
  if constexpr (CPR == 4) return c ^ ((r >> 2) & 3);
  return c ^ ((r ^ (r >> 3)) & 7);
}

// 16 bytes per lane from a buffer straight into LDS: lane l's bytes land at
// dst + 16 * l (dst wave-uniform).
__device__ inline void load_lds16(__amdgpu_buffer_rsrc_t rs, uint8_t* dst, int voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, voff,
                                           0, 0, 0);
}

// Workgroup barrier that the compiler may not move memory accesses across;
// the caller waits for the counters it needs first.
__device__ inline void raw_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Two floats rounded to bfloat16 (nearest, ties to even; NaN stays NaN), low
// half first.
__device__ inline uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{__bf16(lo), __bf16(hi)});
}

// Position t of the order in which an XCD's workgroups take `total` tiles: each
// XCD a contiguous run (workgroups are dispatched round-robin over the 8 XCDs);
// negative past the end.
__device__ inline int xcd_run(int bid, int total) {
  const int xcd = bid & 7, idx = bid >> 3;
  const int base = total >> 3, rem = total & 7;
  if (idx >= base + (xcd < rem ? 1 : 0)) return -1;
  return xcd * base + (xcd < rem ? xcd : rem) + idx;
}

// Tile u of a tiles_m x tiles_n grid: groups of up to 6 tile rows, as even as they
// come, sweeping across the columns. (The 32 tiles an XCD runs at a time then
// share about 6 tile rows and 6 tile columns of operands in its L2; a group of
// one leftover row would share one and 32.)
__device__ inline void tile_of(int u, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int groups = (tiles_m + 5) / 6;
  const int G = (tiles_m + groups - 1) / groups;
  const int per_group = G * tiles_n;
  const int grp = u / per_group;
  const int first_m = grp * G;
  const int gsize = (tiles_m - first_m) < G ? (tiles_m - first_m) : G;
  const int within = u - grp * per_group;
  tm = first_m + within % gsize;
  tn = within / gsize;
}

// One operand of an FP4 product, as a workgroup reads it: `rows` rows, of which K
// step t is 64 bytes at row * ld + t * step; `bytes` of them in all. (Packed rows:
// ld the row length, step 64. With a step's rows together, ld 64: a tile's step is
// then whole cache lines, where 64 bytes of a packed row are half a line and as
// many requests to L2 again.) With block scales, s is
// the step-major scale array at the operand's first row and step, s_step the
// bytes from one K step to the next and s_bytes what may be read from s on.
struct Fp4Operand {
  const uint8_t* q;
  int ld, step, rows, bytes;
  const uint8_t* s;
  int s_step, s_bytes;
};

// FP4 operands of a C::BM x C::BN tile: moves K steps of packed codes into an
// LDS stage, reads the fragments back and multiplies them into acc.
template <class C, bool kMx>
struct Fp4Feed {
  static constexpr int BM = C::BM, BN = C::BN, WN = C::WN, BKB = C::BKB, CPR = C::CPR;
  static constexpr int FM = C::FM, FN = C::FN, NT = C::kThreads;
  static constexpr int SB = C::kStageBytes;
  static_assert(C::kSub == 2, "two 64-code MFMA sub-steps per K step");

  // Operand tiles go straight from global memory to LDS (buffer loads with
  // the LDS destination): one instruction moves 1 KiB, lane l landing at byte
  // 16*l of the block, so the XOR swizzle is applied to the source address.
  // The resource holds the packed matrix size, so rows past M (or N) read as
  // zero codes. A stage is (BM + BN) rows of BKB bytes in 1 KiB blocks (A rows
  // first); wave w moves blocks w, w + W, w + 2W, ...
  static_assert(BKB == 64, "one 1 KiB block is 16 rows of 64 bytes");
  static constexpr int kBlocks = SB / 1024;
  static constexpr int kWaves = NT / kWave;
  static constexpr int kPer = kBlocks / kWaves;
  static_assert(kBlocks % kWaves == 0 && (BM / 16) % kWaves == 0, "even block split");
  static constexpr int kPerA = BM / 16 / kWaves;  // of them A's (the first ones)
  // Block scales (kMx), stored step-major: for K step kt (128 codes, blocks
  // 4kt .. 4kt+3) each row has one 32-bit word at s_step * kt + 4 * row, so
  // the 32 rows of a fragment read 128 contiguous bytes. Lane half h supplies
  // codes 32h .. 32h+31 of each 64-code sub-step, i.e. block 4kt + 2kk + h in
  // sub-step kk: the word shifted right by 8h, byte kk*2 of it picked by the
  // instruction's op_sel. Rows past M (N) take the scales of the last row:
  // their results, zero or NaN with the scale, are not stored. One load serves two
  // fragments (A's two, then B's in pairs): lanes 0..31 read the rows of the
  // first, lanes 32..63 those of the second (64 consecutive rows, 256
  // contiguous bytes), and a lane-half swap (v_permlane32_swap) then gives
  // every lane its row's word of both. The raw words of step kt go into slot
  // kt mod 3 of a register ring, loaded three steps ahead.
  static constexpr int NS = kMx ? FM + FN : 0;  // scale words per step (one per fragment)
  static constexpr int NL = NS / 2;             // scale loads per step
  static_assert(!kMx || (FM % 2 == 0 && FN % 2 == 0), "fragments pair up");
  using Frag = v8i;

  v16f acc[FM][FN];
  __amdgpu_buffer_rsrc_t rsA, rsB, rsSA, rsSB;
  int src_off[kPer];
  int a_row[FM], b_row[FN];
  int sc_off[NL > 0 ? NL : 1];
  int a_step, b_step, sa_step, sb_step;
  int wave, lane, hshift;

  // the tile's first rows of the two operands are m0 and n0
  __device__ inline Fp4Feed(const Fp4Operand& A, const Fp4Operand& B, int m0, int n0, int wave_,
                            int lane_)
      : wave(wave_), lane(lane_), hshift((lane_ >> 5) * 8) {
    const int wm = wave / WN, wn = wave % WN;
    const int a_bytes = A.bytes, b_bytes = B.bytes;
    a_step = A.step;
    b_step = B.step;
    rsA = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A.q), 0, a_bytes, kBufferFlags);
    rsB = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(B.q), 0, b_bytes, kBufferFlags);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = (wave + (j < kPerA ? j : j - kPerA) * kWaves) * 16 + (lane >> 2);
      const int c = (lane & 3) ^ (swz<CPR>(r, 0));  // logical chunk stored at physical lane & 3
      if (j < kPerA)
        src_off[j] = (m0 + r < A.rows) ? (m0 + r) * A.ld + c * 16 : a_bytes;
      else
        src_off[j] = (n0 + r < B.rows) ? (n0 + r) * B.ld + c * 16 : b_bytes;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v16f{};
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) a_row[fm] = wm * (FM * 32) + fm * 32 + (lane & 31);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) b_row[fn] = wn * (FN * 32) + fn * 32 + (lane & 31);
    sa_step = A.s_step;
    sb_step = B.s_step;
    rsSA = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A.s), 0, kMx ? A.s_bytes : 0,
                                             kBufferFlags);
    rsSB = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(B.s), 0, kMx ? B.s_bytes : 0,
                                             kBufferFlags);
    if constexpr (kMx) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int f = 2 * j + (lane >> 5);  // this lane's fragment of load j
        // (a_row and b_row are not indexed here: f differs between lanes)
        const int row = (f < FM ? m0 + wm * (FM * 32) + f * 32 : n0 + wn * (FN * 32) + (f - FM) * 32) +
                        (lane & 31);
        const int lim = f < FM ? A.rows : B.rows;
        sc_off[j] = 4 * (row < lim ? row : lim - 1);
      }
    }
  }

  // (offsets are added as unsigned: that of a row outside the operand is its size,
  // below 2^31, and may pass 2^31 with the step's; it stays past the resource's end)
  __device__ inline void dma(int kt, uint8_t* stage) {
    const uint32_t ka = kt * a_step, kb = kt * b_step;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      uint8_t* const dst = stage + (wave + j * kWaves) * 1024;
      if (j < kPerA)
        load_lds16(rsA, dst, int(uint32_t(src_off[j]) + ka));
      else
        load_lds16(rsB, dst, int(uint32_t(src_off[j]) + kb));
    }
  }

  // fragments of one sub-step (kk) of a stage
  __device__ inline void read_frags(const uint8_t* As, int kk, Frag* af, Frag* bf) {
    const uint8_t* Bs = As + BM * BKB;
    const int c = kk * 2 + (lane >> 5);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int r = a_row[fm];
      const uint4 u = *reinterpret_cast<const uint4*>(As + r * BKB + (swz<CPR>(r, c) << 4));
      af[fm] = v8i{int(u.x), int(u.y), int(u.z), int(u.w), 0, 0, 0, 0};
    }
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
      const int r = b_row[fn];
      const uint4 u = *reinterpret_cast<const uint4*>(Bs + r * BKB + (swz<CPR>(r, c) << 4));
      bf[fn] = v8i{int(u.x), int(u.y), int(u.z), int(u.w), 0, 0, 0, 0};
    }
  }

  // The pipeline's manual vmcnt waits count the stage loads and these in
  // issue order; scheduling barriers keep every group where it is written.
  __device__ inline void load_scales(int kt, uint32_t* dst) {
    if constexpr (kMx) {
#pragma unroll
      for (int j = 0; j < FM / 2; ++j)
        dst[j] = __builtin_amdgcn_raw_buffer_load_b32(rsSA, sc_off[j] + kt * sa_step, 0, 0);
#pragma unroll
      for (int j = FM / 2; j < NL; ++j)
        dst[j] = __builtin_amdgcn_raw_buffer_load_b32(rsSB, sc_off[j] + kt * sb_step, 0, 0);
    }
  }

  // one scale word per fragment from the raw words of a step, shifted to the
  // lane half's block
  __device__ inline void expand(const uint32_t* raw, uint32_t* w) {
    if constexpr (kMx) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const auto sw = __builtin_amdgcn_permlane32_swap(raw[j], raw[j], false, false);
        w[2 * j] = uint32_t(sw[0]) >> hshift;
        w[2 * j + 1] = uint32_t(sw[1]) >> hshift;
      }
    }
  }

  // KK: the sub-step (0 or 1), a template argument so that op_sel is a constant
  template <int KK>
  __device__ inline void mfmas(const Frag* af, const Frag* bf, const uint32_t* sc) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) {
        if constexpr (kMx)
          acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              af[fm], bf[fn], acc[fm][fn], 4, 4, 2 * KK, int(sc[fm]), 2 * KK, int(sc[FM + fn]));
        else
          acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(af[fm], bf[fn], acc[fm][fn],
                                                                        4, 4, 0, 127, 0, 127);
      }
  }
};

// step(kt, 0), step(kt + 1, 1), ... up to S of them, while below end: nested,
// so that no path skips a step and runs a later one.
template <int S, class Step, int I>
__device__ __attribute__((always_inline)) inline void steps_of(const Step& step, int kt, int end,
                                                               std::integral_constant<int, I> i) {
  if constexpr (I < S) {
    if (kt < end) {
      step(kt, i);
      steps_of<S>(step, kt + 1, end, std::integral_constant<int, I + 1>{});
    }
  }
}

// Pipeline over K steps (stage of step s: s mod 3). On entry to step kt the
// first sub-step's fragments of stage kt are in registers. The step reads
// its second sub-step's fragments, issues the first sub-step's MFMAs, then
// waits for its own loads of stage kt+1 (those of kt+2 stay in flight) and
// for its fragment reads, and meets the other waves at a barrier while the
// matrix core works through the queued MFMAs. After the barrier stage kt+1
// is complete and nobody reads stage kt any more, so the loads of step kt+3
// go there; then the second sub-step's MFMAs and the next step's first
// fragment reads. Every wave issues F::kPer loads per step on every path
// (past the last step they repeat it into a stage that is not read).
// With block scales, each step also issues the F::NL scale loads of step kt+3
// after its second sub-step; a step's wait then leaves that step's and the
// previous step's scale loads in flight besides the stage of kt+2.
// On return (nkt >= 1) every load has landed and every wave is done with the
// stages, which may be reused.
template <class F>
__device__ __attribute__((always_inline)) inline void gemm_pipeline(F& f, int nkt, uint8_t* st0,
                                                                    uint8_t* st1, uint8_t* st2) {
  constexpr int kPer = F::kPer, NL = F::NL, NS = F::NS, FM = F::FM, FN = F::FN;
  constexpr int kWaitCnt = waitcnt_vm_lgkm(kPer + 2 * NL, 0);
  static_assert(2 * kPer + 2 * NL < 64, "vmcnt immediate");
  uint32_t sc0[NL > 0 ? NL : 1], sc1[NL > 0 ? NL : 1], sc2[NL > 0 ? NL : 1];
  typename F::Frag a0[FM], b0[FN], a1[FM], b1[FN];
  uint32_t scw[NS > 0 ? NS : 1];
  // a full step inside the main loop (steps kt, kt+1 and kt+2 all exist);
  // sc holds the raw scale words of step kt and is refilled for step kt+3
  auto step = [&](int kt, const uint8_t* cur, const uint8_t* nxt, uint8_t* ldst, uint32_t* sc) {
    f.read_frags(cur, 1, a1, b1);
    f.expand(sc, scw);
    __builtin_amdgcn_sched_barrier(0);
    f.template mfmas<0>(a0, b0, scw);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWaitCnt);
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    f.dma(kt + 3 < nkt ? kt + 3 : nkt - 1, ldst);
    f.template mfmas<1>(a1, b1, scw);
    __builtin_amdgcn_sched_barrier(0);
    f.load_scales(kt + 3 < nkt ? kt + 3 : nkt - 1, sc);
    f.read_frags(nxt, 0, a0, b0);
  };
  // one of the last (up to two) steps: no more loads are issued
  auto tail_step = [&](const uint8_t* cur, const uint8_t* nxt, bool has_next, const uint32_t* sc) {
    f.read_frags(cur, 1, a1, b1);
    f.expand(sc, scw);
    __builtin_amdgcn_sched_barrier(0);
    f.template mfmas<0>(a0, b0, scw);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(0, 0));
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    f.template mfmas<1>(a1, b1, scw);
    __builtin_amdgcn_sched_barrier(0);
    if (has_next) f.read_frags(nxt, 0, a0, b0);
  };
  f.dma(0, st0);
  f.load_scales(0, sc0);
  __builtin_amdgcn_sched_barrier(0);
  f.dma(nkt > 1 ? 1 : nkt - 1, st1);
  f.load_scales(nkt > 1 ? 1 : nkt - 1, sc1);
  __builtin_amdgcn_sched_barrier(0);
  f.dma(nkt > 2 ? 2 : nkt - 1, st2);
  f.load_scales(nkt > 2 ? 2 : nkt - 1, sc2);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(2 * kPer + 2 * NL, 0));  // step 0 landed
  raw_barrier();
  f.read_frags(st0, 0, a0, b0);
  int kt0 = 0;
  for (; kt0 + 3 <= nkt; kt0 += 3) {
    step(kt0, st0, st1, st0, sc0);
    step(kt0 + 1, st1, st2, st1, sc1);
    step(kt0 + 2, st2, st0, st2, sc2);
  }
  if (kt0 < nkt) tail_step(st0, st1, kt0 + 1 < nkt, sc0);
  if (kt0 + 1 < nkt) tail_step(st1, st2, false, sc1);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(0, 0));
  raw_barrier();
}

// The same on S stages, for feeds without block scales whose loads past the last
// step read nothing: S - 1 steps are on their way while one is multiplied. For
// tiles of few rows, whose product is a read of the other operand: the bytes in
// flight set its rate.
template <class F, int S>
__device__ __attribute__((always_inline)) inline void gemm_pipeline_deep(F& f, int nkt,
                                                                         uint8_t* const (&st)[S]) {
  constexpr int kPer = F::kPer, FM = F::FM, FN = F::FN;
  static_assert(F::NL == 0 && (S - 1) * kPer < 64, "vmcnt immediate");
  typename F::Frag a0[FM], b0[FN], a1[FM], b1[FN];
  auto step = [&](int kt, auto i_c) {
    constexpr int i = decltype(i_c)::value;
    f.read_frags(st[i], 1, a1, b1);
    __builtin_amdgcn_sched_barrier(0);
    f.template mfmas<0>(a0, b0, nullptr);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm((S - 2) * kPer, 0));
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    f.dma(kt + S, st[i]);
    f.template mfmas<1>(a1, b1, nullptr);
    __builtin_amdgcn_sched_barrier(0);
    f.read_frags(st[(i + 1) % S], 0, a0, b0);
  };
#pragma unroll
  for (int s = 0; s < S; ++s) {
    f.dma(s, st[s]);
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm((S - 1) * kPer, 0));  // step 0 landed
  raw_barrier();
  f.read_frags(st[0], 0, a0, b0);
  int kt = 0;
  for (; kt + S <= nkt; kt += S) steps_of<S>(step, kt, kt + S, std::integral_constant<int, 0>{});
  steps_of<S>(step, kt, nkt, std::integral_constant<int, 0>{});
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(0, 0));
  raw_barrier();
}

// The same product with the eight waves of a large tile in two groups that take
// turns: waves w and w + 4 share a SIMD, and while one of them multiplies a
// sub-step the other reads its next fragments and issues its loads. Phases are
// separated by workgroup barriers; waves 4..7 pass one more barrier at the start
// (waves 0..3 at the end), which is what shifts them by a phase. With j = 2 kt + kk
// the sub-steps, a wave alternates
//   L_j  reads the fragments of j + 1 (into the other register set); with kk = 0
//        waits for its own loads of step kt + 1, with kk = 1 issues those of
//        step kt + S - 1
//   M_j  multiplies j
// in phases 2j and 2j + 1 (waves 4..7: 2j + 1 and 2j + 2). Step kt + S - 1 goes
// into the stage of step kt - 1: its last fragments, of sub-step 2 kt - 1, were
// waited for by the MFMAs of M_(2 kt - 1), phase 4 kt at the latest, and the loads
// are issued in phase 4 kt + 2 at the earliest. Step kt + 1 is read from phase
// 4 kt + 2 on; every wave has waited for its loads of it by phase 4 kt + 1.
// Steps past the last one are issued as loads that return nothing (F::dma), so
// that the counts stay the same on every path. For feeds without block scales.
template <class F, int S>
__device__ __attribute__((always_inline)) inline void gemm_pipeline_turns(F& f, int nkt,
                                                                          uint8_t* const (&st)[S]) {
  constexpr int kPer = F::kPer, FM = F::FM, FN = F::FN;
  static_assert(F::NL == 0 && (S - 1) * kPer < 64, "vmcnt immediate");
  typename F::Frag a0[FM], b0[FN], a1[FM], b1[FN];
  auto step = [&](int kt, auto i_c) {
    constexpr int i = decltype(i_c)::value;
    constexpr int nxt = (i + 1) % S, prv = (i + S - 1) % S;
    // L, kk = 0
    f.read_frags(st[i], 1, a1, b1);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm((S - 3) * kPer));
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    f.template mfmas<0>(a0, b0, nullptr);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // L, kk = 1
    f.read_frags(st[nxt], 0, a0, b0);
    f.dma(kt + S - 1, st[prv]);
    __builtin_amdgcn_sched_barrier(0);
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    f.template mfmas<1>(a1, b1, nullptr);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    f.dma(s, st[s]);
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm((S - 2) * kPer));  // step 0 landed
  raw_barrier();
  f.read_frags(st[0], 0, a0, b0);
  const bool late = f.wave >= 4;
  if (late) raw_barrier();
  int kt = 0;
  for (; kt + S <= nkt; kt += S) steps_of<S>(step, kt, kt + S, std::integral_constant<int, 0>{});
  steps_of<S>(step, kt, nkt, std::integral_constant<int, 0>{});
  if (!late) raw_barrier();
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm(0, 0));
  raw_barrier();
}

// A finished tile leaves through a wave-private LDS block (the stage buffers
// are free after the pipeline): two 32x32 fragments at a time (one where the
// stages are small) are written in the MFMA layout and read back as rows.
// value(fm, fn, r) is element r of fragment (fm, fn): lanes 0..31 hold 32
// consecutive columns of one row and lanes 32..63 the same columns four rows
// down. emit(row, col, v) takes kVec consecutive elements of one row, row and
// col in the matrix that m0 and n0 index, not yet tested against its size.
template <class C, int kVec, class Value, class Emit>
__device__ __attribute__((always_inline)) inline void emit_tile(uint8_t* st0, uint8_t* st1,
                                                                uint8_t* st2, int wave, int lane,
                                                                int m0, int n0, const Value& value,
                                                                const Emit& emit) {
  constexpr int FM = C::FM, FN = C::FN, kWaves = C::kThreads / kWave;
  constexpr int kPair = FN % 2 == 0 && 3 * (C::kStageBytes / (32 * 72 * 4)) >= kWaves ? 2 : 1;
  // row of a 32 x (32 * kPair) chunk (floats), padded where there is room
  constexpr int kER = 32 * kPair + (3 * (C::kStageBytes / (32 * 40 * 4)) >= kWaves ? 8 : 0);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int col_l = lane & 31;
  // each stage buffer holds the blocks of kEpiPer waves
  constexpr int kEpiPer = C::kStageBytes / (32 * kER * 4);
  static_assert(kEpiPer >= 1 && 3 * kEpiPer >= kWaves, "epilogue blocks fit the stages");
  uint8_t* const ebs = wave < kEpiPer ? st0 : (wave < 2 * kEpiPer ? st1 : st2);
  float* eb = reinterpret_cast<float*>(ebs) + (wave % kEpiPer) * (32 * kER);
  constexpr int kLanes = 32 * kPair / kVec;  // lanes a row
  constexpr int kRows = kWave / kLanes;      // rows a sweep
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int fp = 0; fp < FN; fp += kPair) {
#pragma unroll
      for (int h = 0; h < kPair; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int rl = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
          eb[rl * kER + h * 32 + col_l] = value(fm, fp + h, r);
        }
      const int row_base = m0 + wm * (FM * 32) + fm * 32;
      const int col_base = n0 + wn * (FN * 32) + fp * 32;
#pragma unroll
      for (int it = 0; it < 32 / kRows; ++it) {
        const int rl = it * kRows + lane / kLanes;
        const int cl = (lane % kLanes) * kVec;
        float v[kVec];
#pragma unroll
        for (int i = 0; i < kVec; i += 4) {
          const float4 q = *reinterpret_cast<const float4*>(eb + rl * kER + cl + i);
          v[i] = q.x;
          v[i + 1] = q.y;
          v[i + 2] = q.z;
          v[i + 3] = q.w;
        }
        emit(row_base + rl, col_base + cl, v);
      }
    }
}

// Elements of Out (float, or uint16_t: bfloat16 bits) in 16 bytes.
template <class Out>
constexpr int kOutVec = 16 / int(sizeof(Out));

// kOutVec<Out> consecutive elements to dst, the first `valid` of them; vec:
// dst allows a 16-byte store. bfloat16: one rounding to nearest even, here.
// kStream: non-temporal, so that an output nobody reads soon does not displace
// the operand tiles in L2.
template <bool kStream, class Out>
__device__ __attribute__((always_inline)) inline void store_vec(Out* dst, const float* v, int valid,
                                                                bool vec) {
  if constexpr (sizeof(Out) == 4) {
    const f32x4 u = {v[0], v[1], v[2], v[3]};
    if (vec && valid >= 4) {
      if constexpr (kStream)
        __builtin_nontemporal_store(u, reinterpret_cast<f32x4*>(dst));
      else
        *reinterpret_cast<f32x4*>(dst) = u;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < valid) dst[c] = v[c];
    }
  } else {
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 u = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                     bf16_pair(v[6], v[7])};
    if (vec && valid >= 8) {
      if constexpr (kStream)
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(dst));
      else
        *reinterpret_cast<u32x4*>(dst) = u;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < valid) dst[c] = uint16_t(u[c >> 1] >> (16 * (c & 1)));
    }
  }
}

// Rows of ldy elements from Y on allow 16-byte stores at kOutVec columns.
template <class Out>
__device__ inline bool rows_vec(const Out* Y, int64_t ldy) {
  return (reinterpret_cast<uintptr_t>(Y) & 15) == 0 && ldy % kOutVec<Out> == 0;
}

// The tile's elements to Y (M x N).
template <class C, class Out, class Value>
__device__ __attribute__((always_inline)) inline void store_tile(
    uint8_t* st0, uint8_t* st1, uint8_t* st2, int wave, int lane, int m0, int n0, int M, int N,
    Out* __restrict__ Y, int64_t ldy, const Value& value) {
  const bool vec = rows_vec(Y, ldy);
  emit_tile<C, kOutVec<Out>>(st0, st1, st2, wave, lane, m0, n0, value,
                             [&](int gr, int gc, const float* v) {
                               if (gr < M) store_vec<true>(Y + int64_t(gr) * ldy + gc, v, N - gc, vec);
                             });
}

}  // namespace fp4lin
