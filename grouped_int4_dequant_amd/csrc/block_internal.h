// Internal declarations of the operators of the block around the experts: the
// norms before and after it with its gate and residual, the matrix product with
// bias, activation and residual, and the whole layer for a few tokens, each in 16
// bits. Not installed; the public interface is include/moe_int4.h.
#pragma once

#include "grouped_internal.h"

namespace moe {

// p = o r(o) w_o;  y = scale x + gate p;  n = y r(y) w_n;  r(v) = (mean v^2 + eps)^-1/2
struct NormArgs {
  const uint16_t *o;        // nullable: no block
  int64_t ld_o;
  const void *x;            // nullable: no residual
  int64_t ld_x;
  const void *w_o, *gate, *w_n;  // each nullable
  int32_t w_f32;            // they are fp32, else the operands' type
  int32_t stream_f32;       // x and y are
  int32_t period;           // rows that one row of gate serves
  int32_t T, d;
  float scale, eps;
  void *y;                  // nullable: not wanted
  int64_t ld_y;
  uint16_t *n;              // nullable: not wanted
  int64_t ld_n;
};
// The gradients. Rows are cut into chunks that lie in one gate's rows, or hold whole gates' rows; each
// chunk leaves its column sums in the workspace and a second kernel adds them up.
struct NormGradArgs {
  const void *dy;           // nullable: zeros
  int64_t ld_dy;
  const uint16_t *dn;       // nullable: no norm behind
  int64_t ld_dn;
  const uint16_t *o;        // nullable: no block
  int64_t ld_o;
  const void *y;            // with dn
  int64_t ld_y;
  const void *w_o, *gate, *w_n;
  int32_t w_f32, stream_f32, gates, period, T, d;
  float scale, eps;
  void *dx;                 // nullable: not wanted
  int64_t ld_dx;
  uint16_t *d_o;            // nullable: not wanted
  int64_t ld_do;
  void *dw_o, *dgate, *dw_n;  // each nullable: not wanted
  int32_t g_f32, accumulate;
  float *part;              // workspace: column sums of dw_o, dgate, dw_n, [3][chunks][pitch]
  int64_t pitch;
  int32_t chunk_rows, chunks, per_gate;  // per_gate: chunks of one gate's rows, 0: a chunk holds whole gates
};
// chunk_rows, chunks and per_gate for T rows of which every `period` share a gate
struct NormChunks { int32_t rows, count, per_gate; };
NormChunks norm_chunks(int32_t T, int32_t period);

// dz = act'(pre) dy and its column sums. dz enters the products as 16-bit operands: as the sum of two parts, which hold
// 16 bits of a bf16 dz and 22 of an fp16 one, or of three bf16 parts, which hold it whole (or, if the caller wants that, rounded).
struct ActGradArgs {
  const uint16_t *dy;       // [T][ld_dy], `cols` columns
  int64_t ld_dy;
  const uint16_t *pre;      // [T][ld_pre], N columns; nullable without activation
  int64_t ld_pre;
  int32_t T, N, cols, act;  // cols: N, or N / 2 if gated
  uint16_t *dz;             // [dz_parts][T][N]; nullable without activation
  int32_t dz_parts;         // 1: dz rounded
  int64_t dz_next;          // elements from a part to the next
  float *part;              // nullable: column sums not wanted; [chunks][pitch]
  int64_t pitch;
  int32_t chunk_rows, chunks;
  void *db;                 // [N]
  int32_t g_f32, accumulate;
};
// The parts that the rows of a weight gradient are cut into, where its tiles are too few for the CUs: each part's
// sums go to the workspace in fp32 and are added up in order. wide: whether its operands allow wide tiles.
struct RowParts { int32_t rows, count; };
RowParts weight_parts(int32_t T, int32_t N, int32_t K, bool wide);
struct ColumnChunks { int32_t rows, count; };
ColumnChunks column_chunks(int32_t T, int32_t cols);

// The layer for a few tokens: y[t] = sum_j g_j W_dn (silu(W_g x) * (W_u x)) + shared + add
constexpr int kFewTokens = MOE_MAX_FEW_TOKENS, kFewPairs = MOE_MAX_FEW_PAIRS;
// What the first kernel leaves for the second, at the workspace's begin: the pairs (token, slot) sorted by
// expert and cut into blocks of at most 16 pairs of one expert.
struct FewPlan {
  int32_t blocks;
  int32_t expert[kFewPairs], first[kFewPairs], rows[kFewPairs];  // of each block; first: its first sorted pair
  int32_t pair[kFewPairs];           // token * k + slot
  float gate[kFewPairs];             // by pair
};
struct FewArgs {
  const uint16_t *x;
  int64_t ld_x;
  const float *logits;               // [T][E]
  int32_t T, d, f, f_sh, E, k;
  const uint16_t *gu, *dn, *sh_gu, *sh_dn;  // [E][2f][d], [E][d][f], [2 f_sh][d], [d][f_sh]
  const void *add;                   // nullable, of y's type
  int64_t ld_add;
  void *y;
  int32_t y_f32;
  int64_t ld_y;
  int32_t *topk_ids;                 // nullable [T][k]
  float *topk_w;                     // nullable [T][k]
  FewPlan *plan;                     // workspace
  float *h, *h_sh;                   // workspace: inner values by pair and by token
  int32_t pitch, pitch_sh;           // row pitch of h and h_sh in elements
  int32_t share;                     // gate/up: log2 of the waves that share an item
};
hipError_t launch_few_layer(const FewArgs &a, bool fp16, hipStream_t s);

template <bool Gated>
hipError_t launch_linear(const LinearArgs<Gated> &a, bool fp16, hipStream_t s);
// dz and db, then dx = dz W and dW = dz^T x (each without `out`: not wanted)
// parts: where dW's parts go when dw has more than one (dw.out is dW all the same).
hipError_t launch_linear_grad(const ActGradArgs &c, const DenseArgs &dx, const DenseArgs &dw, float *parts, bool fp16, hipStream_t s);
// The same with dz in more than one part. w, x: fp16 matrices that take part as two bf16 parts (with c.dz in three), and
// where those go; `from` null: they are bf16, or not wanted, or dz is of their type.
struct HalvesArgs {
  const uint16_t *from;     // [rows][ld]
  int64_t ld;
  int32_t rows, cols;
  uint16_t *to;             // [2][rows][cols]
  int64_t next;             // elements from a part to the next
};
hipError_t launch_linear_grad_split(const ActGradArgs &c, const SplitArgs &dx, const SplitArgs &dw, const HalvesArgs &w, const HalvesArgs &x,
                                    float *parts, bool fp16, bool bf16_parts, hipStream_t s);
inline bool is_gated(int32_t act) { return act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU; }

hipError_t launch_norm(const NormArgs &a, bool fp16, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs &a, bool fp16, hipStream_t s);

}  // namespace moe
