// Embedding lookup with scaling, and the gradient of the table.
//
//   out[t] = scale * table[token_t]          zeros for a token outside [0, V)
//   dE[v]  = scale * sum over t with token_t = v of dX[t]   (+ what dE[v] held)
//
// The gradient: the positions are sorted by token (rows.hpp), so every row of the
// table is one thread's sum over its own list, in the order of the positions: no
// atomics, and rows without a token are written in the same pass. A text's few
// frequent tokens have long lists; a list of more than kList positions is cut where
// the sorted positions pass a multiple of kList, each piece is summed by a thread of
// its own into fp32, and a last launch adds a list's pieces in order. So no thread
// adds more than kList rows, however the tokens are distributed.
#include "device_common.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace fp4lin {

namespace {

struct EmbedArgs {
  const void* table;
  int64_t ldt;
  const int32_t* token;
  int32_t V;
  int64_t H;
  float scale;
  void* out;
  int64_t ldo;
  uint32_t items;
};

template <class In, class Out>
__global__ __launch_bounds__(kRowThreads) void embed_kernel(EmbedArgs p, Divisor groups) {
  const Item it = item_of(p.items, groups);
  if (!it.in) return;
  const int32_t t = p.token[it.row];
  const int64_t valid = p.H - it.c;
  by_width(valid, [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    float f[8] = {};
    if (t >= 0 && t < p.V) {
      Vec8<In> v;
      get8<In, kWhole>(static_cast<const typename In::T*>(p.table) + int64_t(t) * p.ldt + it.c, valid, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = In::widen(v.v[i]) * p.scale;
    }
    put8<Out, kWhole>(static_cast<typename Out::T*>(p.out) + int64_t(it.row) * p.ldo + it.c, valid,
                      rounded<Out>(f));
  });
}

__global__ __launch_bounds__(kSortWaves * 64) void embed_sort_kernel(SortArgs p) { sort_body(p); }

constexpr int kList = 32;

struct EmbedBackArgs {
  const void* dX;
  int64_t lddx;
  const int32_t *token, *order, *ends;  // order, ends: of the sort
  int32_t T, V;
  int64_t H;
  float scale;
  int add;
  void* dE;
  int64_t ldde;
  float* part;    // [pieces][2][groups * 8]: of the first list of a piece, of the last
  uint32_t rows;  // items of the table's rows
  uint32_t cuts;  // items of the pieces
};

__device__ inline int32_t list_begin(const EmbedBackArgs& p, int32_t v) { return v > 0 ? p.ends[v - 1] : 0; }

// sum[] += the rows of dX at the sorted positions begin .. end - 1
template <class In, bool kWhole>
__device__ inline void add_rows(const EmbedBackArgs& p, int32_t begin, int32_t end, int64_t c,
                                int64_t valid, float (&sum)[8]) {
  constexpr int U = 4;  // rows in flight
  for (int32_t i = begin; i < end; i += U) {
    Vec8<In> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t t = p.order[i + u < end ? i + u : end - 1];
      get8<In, kWhole>(static_cast<const typename In::T*>(p.dX) + int64_t(t) * p.lddx + c, valid, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u < end) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += In::widen(v[u].v[k]);
      }
  }
}

// scale * sum, or that on top of what is there, to row v
template <class Out, bool kWhole>
__device__ inline void put_row(const EmbedBackArgs& p, int32_t v, int64_t c, int64_t valid,
                               float (&sum)[8]) {
  typename Out::T* const dst = static_cast<typename Out::T*>(p.dE) + int64_t(v) * p.ldde + c;
  if (p.add) {
    Vec8<Out> old;
    get8<Out, kWhole>(dst, valid, old);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = fmaf(sum[k], p.scale, Out::widen(old.v[k]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] *= p.scale;
  }
  put8<Out, kWhole>(dst, valid, rounded<Out>(sum));
}

// The first workgroups take the pieces of long lists, the others the table's rows.
template <class In, class Out>
__global__ __launch_bounds__(kRowThreads) void embed_back_kernel(EmbedBackArgs p, Divisor groups,
                                                                 uint32_t cut_blocks) {
  if (blockIdx.x < cut_blocks) {
    const uint32_t i = blockIdx.x * kRowThreads + threadIdx.x;
    if (i >= p.cuts) return;
    const uint32_t piece = groups(i);
    const int64_t c = int64_t(i - piece * groups.d) * 8, valid = p.H - c;
    const int32_t kept = p.ends[p.V - 1];
    const int32_t a = int32_t(piece) * kList, b = kept - a < kList ? kept : a + kList;
    if (a >= b) return;
    float* const part = p.part + (int64_t(piece) * 2 * groups.d) * 8 + c;
    auto sum_of = [&](int32_t begin, int32_t end, float* dst) {
      float sum[8] = {};
      by_width(valid, [&](auto whole) { add_rows<In, decltype(whole)::value>(p, begin, end, c, valid, sum); });
#pragma unroll
      for (int k = 0; k < 8; ++k) dst[k] = sum[k];
    };
    const int32_t v0 = p.token[p.order[a]], v1 = p.token[p.order[b - 1]];
    const int32_t end0 = p.ends[v0], begin1 = list_begin(p, v1);
    if (end0 - list_begin(p, v0) > kList) sum_of(a, end0 < b ? end0 : b, part);
    if (v1 != v0 && p.ends[v1] - begin1 > kList) sum_of(begin1, b, part + int64_t(groups.d) * 8);
    return;
  }
  const uint64_t i = uint64_t(blockIdx.x - cut_blocks) * kRowThreads + threadIdx.x;
  if (i >= p.rows) return;
  const uint32_t v = groups(uint32_t(i));
  const int64_t c = int64_t(uint32_t(i) - v * groups.d) * 8, valid = p.H - c;
  const int32_t begin = list_begin(p, v), end = p.ends[v];
  if (end - begin > kList || (p.add && begin == end)) return;
  by_width(valid, [&](auto whole) {
    float sum[8] = {};
    add_rows<In, decltype(whole)::value>(p, begin, end, c, valid, sum);
    put_row<Out, decltype(whole)::value>(p, v, c, valid, sum);
  });
}

// The long list that begins in a piece, if one does: its pieces added in order.
template <class Out>
__global__ __launch_bounds__(kRowThreads) void embed_join_kernel(EmbedBackArgs p, Divisor groups) {
  const uint64_t i = uint64_t(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= p.cuts) return;
  const uint32_t piece = groups(uint32_t(i));
  const int64_t c = int64_t(uint32_t(i) - piece * groups.d) * 8, valid = p.H - c;
  const int32_t kept = p.ends[p.V - 1];
  const int32_t a = int32_t(piece) * kList, b = kept - a < kList ? kept : a + kList;
  if (a >= b) return;
  const int32_t v = p.token[p.order[b - 1]];
  const int32_t begin = list_begin(p, v), end = p.ends[v];
  if (begin < a || end - begin <= kList) return;
  const int64_t ld = int64_t(groups.d) * 8;
  // a list that begins with a piece is its first one
  const float* src = p.part + (int64_t(piece) * 2 + (begin > a ? 1 : 0)) * ld + c;
  float sum[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = src[k];
  const int32_t last = (end - 1) / kList;
  constexpr int U = 8;  // pieces in flight
  for (int32_t q = int32_t(piece) + 1; q <= last; q += U) {
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      src = p.part + int64_t(q + u <= last ? q + u : last) * 2 * ld + c;
#pragma unroll
      for (int k = 0; k < 8; ++k) f[u][k] = src[k];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (q + u <= last) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += f[u][k];
      }
  }
  by_width(valid, [&](auto whole) { put_row<Out, decltype(whole)::value>(p, v, c, valid, sum); });
}

}  // namespace

hipError_t launch_embed(const EmbedCall& c, bool table_bf16, bool out_bf16, hipStream_t stream) {
  const Divisor groups(row_groups(c.H));
  const EmbedArgs p{c.table, c.ldt, c.token, int32_t(c.V),           c.H, c.scale,
                    c.out,   c.ldo, uint32_t(c.T) * groups.d};
  return with_type(table_bf16, [&](auto in) {
    return with_type(out_bf16, [&](auto out) {
      embed_kernel<decltype(in), decltype(out)>
          <<<item_blocks(p.items), kRowThreads, 0, stream>>>(p, groups);
      return hipGetLastError();
    });
  });
}

int64_t embed_pieces(int64_t T) { return T > kList ? (T + kList - 1) / kList : 0; }

hipError_t launch_embed_backward(const EmbedCall& c, bool dx_bf16, bool de_bf16, hipStream_t stream) {
  const Divisor groups(row_groups(c.H));
  const SortPlan s = sort_plan(c.V);
  embed_sort_kernel<<<s.blocks, kSortWaves * 64, 0, stream>>>(
      SortArgs{c.token, int32_t(c.T), int32_t(c.V), s.per, c.ends, c.order, nullptr});
  const uint32_t pieces = uint32_t(embed_pieces(c.T));
  const EmbedBackArgs p{c.dX,          c.lddx,  c.token, c.order, c.ends, int32_t(c.T),
                        int32_t(c.V),  c.H,     c.scale, c.add,   c.dE,   c.ldde,
                        c.part,        uint32_t(c.V) * groups.d,  pieces * groups.d};
  const unsigned cut_blocks = item_blocks(p.cuts), row_blocks = item_blocks(p.rows);
  return with_type(de_bf16, [&](auto out) {
    using Out = decltype(out);
    const hipError_t e = with_type(dx_bf16, [&](auto in) {
      embed_back_kernel<decltype(in), Out>
          <<<cut_blocks + row_blocks, kRowThreads, 0, stream>>>(p, groups, cut_blocks);
      return hipGetLastError();
    });
    if (e != hipSuccess || pieces == 0) return e;
    embed_join_kernel<Out><<<cut_blocks, kRowThreads, 0, stream>>>(p, groups);
    return hipGetLastError();
  });
}

}  // namespace fp4lin
