// Launchers behind the C ABI. Arguments are already validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fp4lin.h"

namespace fp4lin {

size_t select_workspace_bytes(bool bf16, int64_t M);
size_t weight_workspace_bytes(int64_t N);

hipError_t launch_outlier_select(const void* A, bool bf16, int64_t M, int64_t K, int64_t lda,
                                 int64_t k, float* tau, int64_t capacity, int32_t* row,
                                 int32_t* col, float* val, int32_t* row_ptr, void* ws,
                                 hipStream_t stream);

// Whole-layer forward, front half: the select of launch_outlier_select (rank
// k, workspace ws of select_workspace_bytes) with the quantization of A
// clamped to tau done by its compaction, and the quantization of W (same
// dtype as A) in launches shared with the select's row kernels. Token-wise:
// sA and sW are float scales and colmax (N words apart from ws) is cleared by
// the select's first pass; micro-scaled (mx): sA and sW are the step-major
// E8M0 arrays and colmax is unused. Any K, alignment and leading dimensions.
struct FrontArgs {
  const void* A;
  bool bf16, mx;
  int64_t M, K, lda, k;
  float* tau;
  int64_t capacity;
  int32_t *row, *col;
  float* val;
  int32_t* row_ptr;
  void* ws;
  uint8_t* Aq;
  int64_t ldq;
  void* sA;
  const void* W;
  int64_t N, ldw;
  uint8_t* Wq;
  void* sW;
  uint32_t* colmax;
};
hipError_t launch_forward_front(const FrontArgs& f, hipStream_t stream);

hipError_t launch_quantize_rows(const void* X, bool bf16, int64_t M, int64_t K, int64_t ldx,
                                const float* tau, uint8_t* Xq, int64_t ldq, float* sX,
                                hipStream_t stream);

hipError_t launch_quantize_weight(const void* W, bool bf16, int64_t K, int64_t N, int64_t ldw,
                                  uint8_t* Wq, int64_t ldq, float* sW, void* ws,
                                  hipStream_t stream);

struct SparseArgs {
  const int32_t* row_ptr;  // nullptr: no compensation term
  const int32_t* col;
  const float* val;
  const void* W;
  bool w_bf16;
  int64_t ldw;
  int64_t w_rows;  // K: rows of W (W is addressed with 32-bit byte offsets)
  int64_t capacity;  // COO entries allocated: bounds the non-zeros (picks the GEMM's schedule)
};

// Y[i, :] += sum over row i's non-zeros of val * W[col, :] (ascending col).
hipError_t launch_sparse_add(const SparseArgs& sp, int64_t M, int64_t N, float* Y, int64_t ldy,
                             hipStream_t stream);

hipError_t launch_fp4_gemm(const uint8_t* Aq, const float* sA, const uint8_t* Bq, const float* sB,
                           int64_t M, int64_t N, int64_t ldq, const SparseArgs& sp, float* Y,
                           int64_t ldy, hipStream_t stream);

// Micro-scaled operands: E2M1 codes with one E8M0 byte per 32 codes along K
// (rows of ldq / 16 bytes). Xs / Ws / As / Bs are those scale rows.
hipError_t launch_quantize_rows_mx(const void* X, bool bf16, int64_t M, int64_t K, int64_t ldx,
                                   const float* tau, uint8_t* Xq, int64_t ldq, uint8_t* Xs,
                                   hipStream_t stream);
hipError_t launch_quantize_cols_mx(const void* W, bool bf16, int64_t K, int64_t N, int64_t ldw,
                                   uint8_t* Wq, int64_t ldq, uint8_t* Ws, hipStream_t stream);
hipError_t launch_fp4_gemm_mx(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                              const uint8_t* Bs, int64_t M, int64_t N, int64_t ldq,
                              const SparseArgs& sp, float* Y, int64_t ldy, hipStream_t stream);

// Products grouped by expert (experts.hip). experts_steps: the K steps (128
// rows) of a reduction over each expert's own rows, for any split of M rows.
int64_t experts_steps(int64_t E, int64_t M);
hipError_t launch_experts_quantize_weight_mx(const void* W, bool bf16, int64_t E, int64_t K,
                                             int64_t N, int64_t ldw, uint8_t* Wq, int64_t ldq,
                                             uint8_t* Ws, hipStream_t stream);
// The operands of the products below, in the order of experts.hip (a K step's
// rows together), both of a product in one launch.
hipError_t launch_experts_quantize_rows(const void* A, bool bf16, int64_t M, int64_t K, int64_t lda,
                                        uint8_t* Aq, uint8_t* As, hipStream_t stream);
hipError_t launch_experts_quantize_forward(const void* A, const void* W, bool bf16, int64_t E,
                                           int64_t M, int64_t K, int64_t N, int64_t lda,
                                           int64_t ldw, uint8_t* Aq, uint8_t* As, uint8_t* Wq,
                                           uint8_t* Ws, hipStream_t stream);
hipError_t launch_experts_quantize_dgrad(const void* dY, const void* W, bool bf16, int64_t E,
                                         int64_t M, int64_t K, int64_t N, int64_t lddy, int64_t ldw,
                                         uint8_t* Dq, uint8_t* Ds, uint8_t* Wq, uint8_t* Ws,
                                         hipStream_t stream);
hipError_t launch_experts_quantize_wgrad(const void* A, const void* dY, bool bf16,
                                         const int32_t* row_end, int64_t E, int64_t M, int64_t K,
                                         int64_t N, int64_t lda, int64_t lddy, uint8_t* Aq,
                                         uint8_t* As, uint8_t* Dq, uint8_t* Ds,
                                         hipStream_t stream);
// M rows against N columns of each expert (forward, dgrad, apply); packed: the
// weights are in packed rows, as launch_experts_quantize_weight_mx leaves them.
hipError_t launch_experts_rows(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                               const uint8_t* Bs, const int32_t* row_end, int64_t E, int64_t M,
                               int64_t N, int64_t ldq, bool packed, void* Y, bool y_bf16,
                               int64_t ldy, hipStream_t stream);
// The same for so few rows that the product quantizes them itself.
bool experts_fused(int64_t M, int64_t K);
hipError_t launch_experts_fused(const void* A, bool bf16, int64_t lda, const uint8_t* Bq,
                                const uint8_t* Bs, const int32_t* row_end, int64_t E, int64_t M,
                                int64_t K, int64_t N, int64_t ldq, void* Y, bool y_bf16,
                                int64_t ldy, hipStream_t stream);
hipError_t launch_experts_wgrad(const uint8_t* Aq, const uint8_t* As, const uint8_t* Bq,
                                const uint8_t* Bs, const int32_t* row_end, int64_t E, int64_t M,
                                int64_t K, int64_t N, void* dW, bool w_bf16, int64_t ldw,
                                hipStream_t stream);

// Head loss (head.hip). The plan follows from sizes and strides alone.
struct HeadPlan {
  bool pack_x, pack_w;       // operands copied into the workspace, padded
  bool step_x;               // X copied with a K step's rows together
  int64_t ldx, ldw;          // row strides the products use
  int64_t x_bytes, w_bytes;  // of the copies
  int64_t parts;             // (m, s) pairs a row
  int64_t piece;             // vocabulary columns a piece of the backward
  int64_t ldg;               // row stride of G
  int64_t slices, ldp;       // dX: reduction slices, row stride of their arrays
};
HeadPlan head_plan(bool bf16, bool backward, int64_t T, int64_t H, int64_t V, bool by_vocab,
                   int64_t ldx, int64_t ldw);

struct HeadCall {
  const void *X, *W;
  int64_t T, H, V, ldx, ldw;
  bool by_vocab;
  const int32_t* target;
  // workspace
  void *packed_x, *packed_w, *part, *G;
  float *tlogit, *acc, *top;
  // forward
  float *loss, *lse_out;
  // backward
  const float *lse, *dloss;
  void *dX, *dW;
  int64_t lddx, lddw;
  // distillation (k > 0): a teacher's k entries a row; target is then `kept`
  int64_t k;
  const int32_t* index;
  const void* teacher;
  bool teacher_bf16;
  float inv_temperature;
  void *teacher_entry, *teacher_sums;
  uint16_t* teacher_first;
  int32_t* kept;
  float* tdot;

  bool distill() const { return k > 0; }
};
hipError_t launch_head_loss(const HeadCall& c, bool bf16, const HeadPlan& h, hipStream_t stream);
hipError_t launch_head_loss_backward(const HeadCall& c, bool bf16, const HeadPlan& h,
                                     hipStream_t stream);

// Rows of tokens to their experts and back (route.hip): T tokens, k slots each.
struct RouteCall {
  int64_t T, k, E, H;
  // dispatch
  const void* X;
  int64_t ldx;
  const int32_t* expert;
  void* Xs;
  int64_t ldxs;
  int32_t *row_end_out, *slot_row_out;
  // the way back
  const int32_t *slot_row, *row_end;
  const float* weight;  // may be NULL
  const void* Y;
  int64_t ldy;
  const void* residual;  // may be NULL
  int64_t ldr;
  void* out;
  int64_t ldo;
  // and its gradient
  const void* dout;
  int64_t lddo;
  void* dY;
  int64_t lddy;
  float* dweight;  // may be NULL
};
hipError_t launch_experts_dispatch(const RouteCall& c, bool bf16, hipStream_t stream);
hipError_t launch_experts_combine(const RouteCall& c, bool y_bf16, bool out_bf16, hipStream_t stream);
hipError_t launch_experts_combine_backward(const RouteCall& c, bool y_bf16, bool dout_bf16,
                                           bool dy_bf16, hipStream_t stream);

// Embedding (embed.hip). embed_pieces: pieces of up to T positions; the gradient
// keeps two fp32 rows of each, H rounded up to 8.
struct EmbedCall {
  int64_t T, V, H;
  const int32_t* token;
  float scale;
  // lookup
  const void* table;
  int64_t ldt;
  void* out;
  int64_t ldo;
  // gradient
  const void* dX;
  int64_t lddx;
  bool add;
  void* dE;
  int64_t ldde;
  void* order;  // T pairs of int32
  int32_t* ends;
  float* part;
};
hipError_t launch_embed(const EmbedCall& c, bool table_bf16, bool out_bf16, hipStream_t stream);
int64_t embed_pieces(int64_t T);
hipError_t launch_embed_backward(const EmbedCall& c, bool dx_bf16, bool de_bf16, hipStream_t stream);

// Gradient norm and clipping (clip.hip). clip_parts: partial sums that `count`
// tensors of `elements` elements in all can need; ws holds two doubles more.
int64_t clip_parts(int64_t count, int64_t elements);
hipError_t launch_clip(const fp4lin_grad* grads, int64_t count, int64_t elements, bool clip,
                       float max_norm, float* norm, void* ws, hipStream_t stream);

}  // namespace fp4lin
