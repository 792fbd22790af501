// Internal declarations of the 16-bit operators: products grouped by expert
// and their gradients, the weighted combine of expert rows and its gradient,
// and low-rank adapters beside a shared projection. Not installed; the public
// interface is include/moe_int4.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_int4.h"

namespace moe {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch holds fewer than 2^32 threads along a dimension of its grid; the
// launch functions below answer hipErrorInvalidConfiguration to more.
inline bool grid_fits(int64_t blocks, int threads) { return blocks * threads < (int64_t)1 << 32; }

// out[i][j] = sum_r L[i][r] * R[j][r], per group. Which of the two operands
// lies with r contiguous in memory, and which dimension the groups cut, is
// the mode:
//   kFwd    i = sorted row, j = output column n, r = input column k
//           (L = A rows through a_row, R = W_e)
//   kDgrad  i = sorted row, j = k, r = n (L = dC rows, R = W_e read across its rows)
//   kWgrad  i = n, j = k, r = sorted row (both read across their rows)
enum GroupedMode { kFwd = 0, kDgrad = 1, kWgrad = 2 };

struct GroupedArgs {
  const uint16_t *rows;     // A (forward, weight gradient) or dC (input gradient)
  int64_t ld_rows;
  const int32_t *a_row;     // nullable: row of `rows` for each sorted row
  int32_t a_rows;           // rows of A that exist
  const uint16_t *w;        // W [G][N][K] (forward, input gradient) or dC (weight gradient)
  int64_t ld_w;             // K, or dC's row stride
  const int32_t *offsets;   // [G+1]
  int32_t G, P, N, K;
  void *out;
  int64_t ld_out;
  int32_t out_f32;          // out is fp32, else the operands' type
  int32_t accumulate;       // fp32 out only: out += result
  int32_t vec;              // every 16-byte unit of the operands is aligned and whole
  int32_t wide;             // 31-bit byte offsets reach every operand of the wide tiles
  int32_t vec_out;          // four consecutive outputs may be stored at once
};

hipError_t launch_grouped(const GroupedArgs &a, GroupedMode mode, bool fp16, hipStream_t s);

// y[t] = sum_j w[t][j] o[pos[t][j]] + add[t]
struct CombineRowsArgs {
  const uint16_t *o;
  int64_t ld_o;
  int32_t P;
  const int32_t *pos;       // [T][k]; a value outside [0, P) is no row
  const float *w;           // nullable: ones
  int32_t T, k, d;
  const void *add;          // nullable
  int32_t add_f32;
  int64_t ld_add;
  void *y;
  int32_t y_f32;
  int64_t ld_y;
  int32_t vec;              // eight consecutive values of every array may be read or stored at once
};
// d_o[pos[t][j]] = w[t][j] dy[t];  dw[t][j] = <dy[t], o[pos[t][j]]>
struct CombineRowsGradArgs {
  const uint16_t *dy, *o;   // o nullable with dw
  int64_t ld_dy, ld_o;
  int32_t P;
  const int32_t *pos;
  const float *w;           // nullable: ones
  int32_t T, k, d;
  uint16_t *d_o;            // nullable
  int64_t ld_do;
  float *dw;                // nullable
  int32_t vec;
};
hipError_t launch_combine_rows(const CombineRowsArgs &a, bool fp16, hipStream_t s);
hipError_t launch_combine_rows_grad(const CombineRowsGradArgs &a, bool fp16, hipStream_t s);

// Adapters: y[t] = base[t] + scale_a B_a (A_a x[t]) over rows sorted by adapter.
constexpr int kMaxRank = MOE_MAX_ADAPTER_RANK;
inline int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

struct AdapterArgs {
  const uint16_t *x;        // [T][ld_x]
  int64_t ld_x;
  int32_t T, K, N, r, n;
  const uint16_t *A;        // [n][r][K]
  const uint16_t *B;        // [n][N][r]
  const float *scale;       // nullable: ones
  const int32_t *rows;      // [T] row of each sorted place; a value outside [0, T) is no row
  const int32_t *offsets;   // [n+1]; places from offsets[n] on have no adapter
  const void *base;         // nullable: zeros
  int64_t ld_base;
  void *y;
  int32_t y_f32;
  int64_t ld_y;
  int32_t vec_x, vec_y, vec_b;  // 16-byte units of x and A, of base and y, of B are aligned
};
struct AdapterGradArgs {
  const uint16_t *dy, *x;
  int64_t ld_dy, ld_x;
  int32_t T, K, N, r, n;
  const uint16_t *A, *B;
  const float *scale;
  const int32_t *rows, *offsets;
  const void *dx_base;      // nullable: zeros
  int64_t ld_dx_base;
  void *dx;                 // nullable: not wanted
  int32_t dx_f32;
  int64_t ld_dx;
  void *dA, *dB;            // each nullable: not wanted
  int32_t g_f32, accumulate;
  float *g, *h;             // workspace, fp32 [T][16 rank_tiles(r)] by sorted place: scale B^T dy and scale A x
  int32_t vec_x, vec_dy, vec_dx, vec_b;
  int32_t vec_da;           // four consecutive values of dA may be stored at once
};
hipError_t launch_adapter_plan(const int32_t *row_adapter, int32_t T, int32_t n, int32_t *rows, int32_t *offsets, hipStream_t s);
hipError_t launch_adapter(const AdapterArgs &a, bool fp16, hipStream_t s);
hipError_t launch_adapter_grad(const AdapterGradArgs &a, bool fp16, hipStream_t s);

}  // namespace moe
