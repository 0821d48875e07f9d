// Rows of tokens to their experts and back.
//
// T tokens go to k experts each; slot i = t * k + j is token t's j-th. The slots
// are sorted by expert, stably; slots whose expert lies outside [0, E) come last.
//
//   dispatch          Xs[row(t, j)] = X[t], zeros for a slot without an expert
//   combine           out[t] = residual[t] + sum_j w[t, j] * Y[row(t, j)]
//   combine_backward  dY[row(t, j)] = w[t, j] * dout[t]
//                     dw[t, j] = <dout[t], Y[row(t, j)]>
//
// Every kernel goes by token, not by row: a token's row is read once, whatever k,
// and its slots' rows are reached through slot_row, whose sums are then over a
// token's own few rows in slot order. No atomics. All sums are fp32; what is
// stored in bfloat16 is rounded once.
#include "device_common.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace fp4lin {

namespace {

__global__ __launch_bounds__(kSortWaves * 64) void route_sort_kernel(SortArgs p) { sort_body(p); }

// Rows that an expert has made: those below row_end's last entry, clamped.
__device__ inline int32_t rows_made(const int32_t* row_end, int32_t E, int32_t M) {
  const int32_t n = row_end[E - 1];
  return n < 0 ? 0 : n < M ? n : M;
}

struct DispatchArgs {
  const void* X;
  int64_t ldx;
  void* Xs;
  int64_t ldxs;
  const int32_t* expert;  // dispatch_few_kernel only
  int32_t *slot_row, *row_end;
  int32_t k, E, M;
  int64_t H;
  uint32_t items;
};

template <class In>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(DispatchArgs p, Divisor groups) {
  const Item it = item_of(p.items, groups);
  if (!it.in) return;
  const int64_t valid = p.H - it.c;
  by_width(valid, [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    Vec8<In> v;
    get8<In, kWhole>(static_cast<const typename In::T*>(p.X) + int64_t(it.row) * p.ldx + it.c, valid, v);
    const int32_t made = rows_made(p.row_end, p.E, p.M);
    const int32_t* const rows = p.slot_row + int64_t(it.row) * p.k;
    for (int32_t j = 0; j < p.k; ++j) {
      const int32_t r = rows[j];
      put8<In, kWhole>(static_cast<typename In::T*>(p.Xs) + int64_t(r) * p.ldxs + it.c, valid,
                       r < made ? v : Vec8<In>{});
    }
  });
}

// A few slots (up to kFewSlots) sorted and moved in one launch: every workgroup
// has all keys in shared memory and finds the places of its own tokens' slots by
// counting those that come before, 64 a step by ballot. Workgroup b takes token
// b / parts and a part of its columns; the ends of the experts' rows are spread over
// all waves.
constexpr int kFewSlots = 1024;

template <class In>
__global__ __launch_bounds__(kRowThreads) void dispatch_few_kernel(DispatchArgs p, int parts) {
  __shared__ int32_t key[kFewSlots];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = blockIdx.x / parts, part = blockIdx.x - token * parts;
  const int64_t c = (int64_t(part) * kRowThreads + threadIdx.x) * 8, valid = p.H - c;
  const typename In::T* const x = static_cast<const typename In::T*>(p.X) + int64_t(token) * p.ldx;
  Vec8<In> v;
  // on its way while the slots are sorted
  if (valid > 0)
    by_width(valid, [&](auto whole) { get8<In, decltype(whole)::value>(x + c, valid, v); });
  const int steps = (p.M + 63) / 64;
  for (int i = threadIdx.x; i < steps * 64; i += kRowThreads) {
    const int32_t e = i < p.M ? p.expert[i] : 0;
    key[i] = i >= p.M ? p.E + 1 : e >= 0 && e < p.E ? e : p.E;
  }
  __syncthreads();
  const int waves = gridDim.x * (kRowThreads / 64);
  for (int e = blockIdx.x * (kRowThreads / 64) + wave; e < p.E; e += waves) {
    int32_t n = 0;
    for (int s = 0; s < steps; ++s) n += __builtin_popcountll(__ballot(key[s * 64 + lane] <= e));
    if (lane == 0) p.row_end[e] = n;
  }
  for (int j = 0; j < p.k; ++j) {
    const int slot = token * p.k + j;
    const int32_t mine = key[slot];
    int32_t r = 0;
    for (int s = 0; s < steps; ++s) {
      const int i = s * 64 + lane;
      const int32_t other = key[i];
      r += __builtin_popcountll(__ballot(other < mine || (other == mine && i < slot)));
    }
    if (part == 0 && threadIdx.x == 0) p.slot_row[slot] = r;
    if (valid > 0)
      by_width(valid, [&](auto whole) {
        put8<In, decltype(whole)::value>(
            static_cast<typename In::T*>(p.Xs) + int64_t(r) * p.ldxs + c, valid,
            mine < p.E ? v : Vec8<In>{});
      });
  }
}

struct CombineArgs {
  const void* Y;
  int64_t ldy;
  const int32_t *slot_row, *row_end;
  const float* weight;   // NULL: ones
  const void* residual;  // NULL: zeros; of the output's type
  int64_t ldr;
  void* out;
  int64_t ldo;
  int32_t k, E, M;
  int64_t H;
  uint32_t items;
};

constexpr int kSlots = 4;  // of a token, their rows read together

template <class In, class Out>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(CombineArgs p, Divisor groups) {
  const Item it = item_of(p.items, groups);
  if (!it.in) return;
  const int64_t valid = p.H - it.c;
  by_width(valid, [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    Vec8<Out> res{};
    if (p.residual != nullptr)
      get8<Out, kWhole>(
          static_cast<const typename Out::T*>(p.residual) + int64_t(it.row) * p.ldr + it.c, valid, res);
    const int32_t made = rows_made(p.row_end, p.E, p.M);
    float sum[8] = {};
    const int64_t slot0 = int64_t(it.row) * p.k;
    for (int32_t j0 = 0; j0 < p.k; j0 += kSlots) {
      Vec8<In> v[kSlots];
      float w[kSlots];
      bool has[kSlots];
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const int32_t j = j0 + u < p.k ? j0 + u : p.k - 1;
        const int32_t r = p.slot_row[slot0 + j];
        has[u] = j0 + u < p.k && r >= 0 && r < made;
        w[u] = p.weight != nullptr ? p.weight[slot0 + j] : 1.0f;
        if (has[u])
          get8<In, kWhole>(static_cast<const typename In::T*>(p.Y) + int64_t(r) * p.ldy + it.c, valid,
                           v[u]);
      }
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (has[u]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[u], In::widen(v[u].v[i]), sum[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += Out::widen(res.v[i]);
    put8<Out, kWhole>(static_cast<typename Out::T*>(p.out) + int64_t(it.row) * p.ldo + it.c, valid,
                      rounded<Out>(sum));
  });
}

struct CombineBackArgs {
  const void* dout;
  int64_t lddo;
  const void* Y;  // read for dweight only
  int64_t ldy;
  const int32_t *slot_row, *row_end;
  const float* weight;  // NULL: ones
  void* dY;
  int64_t lddy;
  float* dweight;  // NULL: not wanted
  int32_t T, k, E, M;
  int64_t H;
};

// kPer threads a token. A row of dout is read once for kSlots slots.
template <class In, class D, class Out, int kPer>
__global__ __launch_bounds__(kRowThreads) void combine_back_kernel(CombineBackArgs p) {
  constexpr int kTokens = kRowThreads / kPer, kParts = kPer > 64 ? kPer / 64 : 1;
  __shared__ float part[kParts][kSlots];
  const int t = threadIdx.x % kPer;
  const int64_t token = int64_t(blockIdx.x) * kTokens + threadIdx.x / kPer;
  const bool in = token < p.T;
  const int32_t made = rows_made(p.row_end, p.E, p.M);
  const typename D::T* const d = static_cast<const typename D::T*>(p.dout) + (in ? token : 0) * p.lddo;
  const int64_t slot0 = (in ? token : 0) * p.k;
  const bool dots = p.dweight != nullptr;
  for (int32_t j0 = 0; j0 < p.k; j0 += kSlots) {
    int32_t r[kSlots];
    float w[kSlots], dot[kSlots] = {};
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      const int32_t j = j0 + u < p.k ? j0 + u : p.k - 1;
      r[u] = p.slot_row[slot0 + j];
      if (!in || j0 + u >= p.k || r[u] >= p.M) r[u] = -1;
      w[u] = p.weight != nullptr ? p.weight[slot0 + j] : 1.0f;
    }
    for (int64_t c = int64_t(t) * 8; c < p.H; c += int64_t(kPer) * 8) {
      const int64_t valid = p.H - c;
      by_width(valid, [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        Vec8<D> g;
        get8<D, kWhole>(d + c, valid, g);
        Vec8<In> y[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if (dots && r[u] >= 0 && r[u] < made)
            get8<In, kWhole>(static_cast<const typename In::T*>(p.Y) + int64_t(r[u]) * p.ldy + c, valid,
                             y[u]);
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          if (r[u] < 0) continue;
          float o[8] = {};
          if (r[u] < made) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float gi = D::widen(g.v[i]);
              o[i] = w[u] * gi;
              if (dots) dot[u] = fmaf(gi, In::widen(y[u].v[i]), dot[u]);
            }
          }
          put8<Out, kWhole>(static_cast<typename Out::T*>(p.dY) + int64_t(r[u]) * p.lddy + c, valid,
                            rounded<Out>(o));
        }
      });
    }
    if (!dots) continue;
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
#pragma unroll
      for (int off = (kPer < 64 ? kPer : 64) / 2; off >= 1; off >>= 1)
        dot[u] += __shfl_xor(dot[u], off, kWave);
    }
    if constexpr (kParts > 1) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int u = 0; u < kSlots; ++u) part[threadIdx.x >> 6][u] = dot[u];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        dot[u] = part[0][u];
#pragma unroll
        for (int q = 1; q < kParts; ++q) dot[u] += part[q][u];
      }
    }
    if (t == 0 && in) {
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (j0 + u < p.k) p.dweight[slot0 + j0 + u] = dot[u];
    }
  }
}

template <class In>
hipError_t run_dispatch(const RouteCall& c, hipStream_t stream) {
  const int64_t M = c.T * c.k;
  DispatchArgs p{c.X,        c.ldx,       c.Xs,       c.ldxs, c.expert, c.slot_row_out, c.row_end_out,
                 int32_t(c.k), int32_t(c.E), int32_t(M), c.H,    0};
  if (M <= kFewSlots && M > 0) {
    const int64_t parts = (row_groups(c.H) + kRowThreads - 1) / kRowThreads;
    dispatch_few_kernel<In><<<unsigned(c.T * parts), kRowThreads, 0, stream>>>(p, int(parts));
    return hipGetLastError();
  }
  const SortPlan s = sort_plan(c.E);
  route_sort_kernel<<<s.blocks, kSortWaves * 64, 0, stream>>>(
      SortArgs{c.expert, int32_t(M), int32_t(c.E), s.per, c.row_end_out, nullptr, c.slot_row_out});
  if (M > 0) {
    const Divisor groups(row_groups(c.H));
    p.items = uint32_t(c.T) * groups.d;
    dispatch_kernel<In><<<item_blocks(p.items), kRowThreads, 0, stream>>>(p, groups);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_dispatch(const RouteCall& c, bool bf16, hipStream_t stream) {
  return with_type(bf16, [&](auto in) { return run_dispatch<decltype(in)>(c, stream); });
}

hipError_t launch_experts_combine(const RouteCall& c, bool y_bf16, bool out_bf16, hipStream_t stream) {
  const Divisor groups(row_groups(c.H));
  const CombineArgs p{c.Y,          c.ldy,        c.slot_row,         c.row_end, c.weight,
                      c.residual,   c.ldr,        c.out,              c.ldo,     int32_t(c.k),
                      int32_t(c.E), int32_t(c.T * c.k), c.H,          uint32_t(c.T) * groups.d};
  return with_type(y_bf16, [&](auto in) {
    return with_type(out_bf16, [&](auto out) {
      combine_kernel<decltype(in), decltype(out)>
          <<<item_blocks(p.items), kRowThreads, 0, stream>>>(p, groups);
      return hipGetLastError();
    });
  });
}

hipError_t launch_experts_combine_backward(const RouteCall& c, bool y_bf16, bool dout_bf16,
                                           bool dy_bf16, hipStream_t stream) {
  const CombineBackArgs p{c.dout,  c.lddo,    c.Y,          c.ldy,        c.slot_row,   c.row_end,
                          c.weight, c.dY,     c.lddy,       c.dweight,    int32_t(c.T), int32_t(c.k),
                          int32_t(c.E), int32_t(c.T * c.k), c.H};
  return with_type(y_bf16, [&](auto in) {
    return with_type(dout_bf16, [&](auto d) {
      return with_type(dy_bf16, [&](auto out) {
        auto go = [&](auto per_c) {
          constexpr int kPer = decltype(per_c)::value;
          const unsigned blocks = unsigned((c.T + kRowThreads / kPer - 1) / (kRowThreads / kPer));
          combine_back_kernel<decltype(in), decltype(d), decltype(out), kPer>
              <<<blocks, kRowThreads, 0, stream>>>(p);
          return hipGetLastError();
        };
        if (c.H <= 128) return go(std::integral_constant<int, 16>{});
        if (c.H <= 512) return go(std::integral_constant<int, 64>{});
        return go(std::integral_constant<int, 256>{});
      });
    });
  });
}

}  // namespace fp4lin
