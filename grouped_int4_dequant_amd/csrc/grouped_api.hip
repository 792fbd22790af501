// C ABI of the 16-bit operators: argument validation and launches. Every
// check runs on the host before anything is enqueued; nothing here reads device
// memory, allocates or synchronises.

#include "grouped_internal.h"

#include <limits.h>

using namespace moe;

namespace {

// Row and column counts in 32 bits leave room for a tile beyond the last one.
constexpr int32_t kMaxExtent = 1 << 30;

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool is16(int32_t t) { return t == MOE_BF16 || t == MOE_FP16; }
// an output type beside operands of type t: t itself, or fp32
bool out_type(int32_t o, int32_t t) { return o == t || o == MOE_FP32; }
size_t size_of(int32_t t) { return t == MOE_FP32 ? 4 : 2; }
bool typed(const void *p, int32_t t) { return aligned(p, size_of(t)); }
// 16-byte units of rows of `width` 16-bit elements are aligned and whole
bool units(const void *p, int64_t ld, int64_t width) { return aligned(p, 16) && ld % 8 == 0 && width % 8 == 0; }
// 16-byte runs of rows of elements of type t are aligned
bool runs(const void *p, int32_t t, int64_t ld) { return aligned(p, 16) && ld * size_of(t) % 16 == 0; }

// The wide-tile kernel reads its operands through 31-bit byte offsets: from
// the start of A where rows are gathered, of the tile's rows where they are
// consecutive, of a group's rows for the weight gradient, and of a group's weights.
bool wide_tiles(const GroupedArgs &a, GroupedMode mode) {
  const int64_t limit = (int64_t)1 << 30;  // elements
  if (!a.vec || a.a_rows < 1) return false;
  if ((int64_t)a.N * a.K >= limit || 256 * a.ld_rows >= limit) return false;
  if (mode == kWgrad) return a.P * a.ld_w < limit && a.a_rows * a.ld_rows < limit;
  return !a.a_row || a.a_rows * a.ld_rows < limit;
}

int status(hipError_t e) {
  return e == hipSuccess ? MOE_OK : e == hipErrorInvalidConfiguration ? MOE_EUNSUPPORTED : MOE_EHIP;
}

int check_groups(int32_t dtype, int32_t out, const int32_t *offsets, int32_t G, int32_t P, int32_t N, int32_t K) {
  if (!is16(dtype) || !out_type(out, dtype)) return MOE_EINVAL;
  if (!offsets || !aligned(offsets, 4) || G < 1 || P < 0 || N < 1 || K < 1) return MOE_EINVAL;
  if (G > MOE_MAX_EXPERTS || P > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_adapter(int32_t dtype, const uint16_t *x, int64_t ld_x, int32_t T, int32_t K, int32_t N, int32_t r, int32_t n,
                  const uint16_t *A, const uint16_t *B, const float *scale, const int32_t *rows, const int32_t *offsets) {
  if (!is16(dtype) || T < 0 || K < 1 || N < 1 || r < 1 || n < 1) return MOE_EINVAL;
  if (!A || !B || !offsets || !aligned(A, 2) || !aligned(B, 2) || !aligned(offsets, 4) || !aligned(scale, 4)) return MOE_EINVAL;
  if (T > 0 && (!x || !rows || !aligned(x, 2) || !aligned(rows, 4) || ld_x < K)) return MOE_EINVAL;
  if (r > MOE_MAX_ADAPTER_RANK || n > MOE_MAX_ADAPTERS || T > MOE_MAX_TOKENS || K > kMaxExtent || N > kMaxExtent) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_gemm(int32_t dtype, const void *A, int64_t lda, int32_t a_rows, const int32_t *a_row,
                     const int32_t *offsets, int32_t G, int32_t P, int32_t N, int32_t K, const void *W, void *C,
                     int32_t c_dtype, int64_t ldc, hipStream_t stream) {
  const int st = check_groups(dtype, c_dtype, offsets, G, P, N, K);
  if (st != MOE_OK) return st;
  if (a_rows < 0 || lda < K || ldc < N) return MOE_EINVAL;
  if (P == 0) return MOE_OK;
  if ((!A && a_rows > 0) || !W || !C || !typed(A, dtype) || !typed(W, dtype) || !typed(C, c_dtype) || !aligned(a_row, 4)) return MOE_EINVAL;
  GroupedArgs a{};
  a.rows = static_cast<const uint16_t *>(A);
  a.ld_rows = lda;
  a.a_row = a_row;
  a.a_rows = a_rows;
  a.w = static_cast<const uint16_t *>(W);
  a.ld_w = K;
  a.offsets = offsets;
  a.G = G; a.P = P; a.N = N; a.K = K;
  a.out = C;
  a.ld_out = ldc;
  a.out_f32 = c_dtype == MOE_FP32;
  a.vec = units(A, lda, K) && units(W, K, K);
  a.wide = wide_tiles(a, kFwd);
  a.vec_out = runs(C, c_dtype, ldc) && N % 4 == 0;
  return status(launch_grouped(a, kFwd, dtype == MOE_FP16, stream));
}

int moe_grouped_gemm_dgrad(int32_t dtype, const void *dC, int64_t lddc, const int32_t *offsets, int32_t G, int32_t P,
                           int32_t N, int32_t K, const void *W, void *dA, int32_t da_dtype, int64_t ldda,
                           hipStream_t stream) {
  const int st = check_groups(dtype, da_dtype, offsets, G, P, N, K);
  if (st != MOE_OK) return st;
  if (lddc < N || ldda < K) return MOE_EINVAL;
  if (P == 0) return MOE_OK;
  if (!dC || !W || !dA || !typed(dC, dtype) || !typed(W, dtype) || !typed(dA, da_dtype)) return MOE_EINVAL;
  GroupedArgs a{};
  a.rows = static_cast<const uint16_t *>(dC);
  a.ld_rows = lddc;
  a.a_rows = P;
  a.w = static_cast<const uint16_t *>(W);
  a.ld_w = K;
  a.offsets = offsets;
  a.G = G; a.P = P; a.N = N; a.K = K;
  a.out = dA;
  a.ld_out = ldda;
  a.out_f32 = da_dtype == MOE_FP32;
  a.vec = units(dC, lddc, N) && units(W, K, K);
  a.wide = wide_tiles(a, kDgrad);
  a.vec_out = runs(dA, da_dtype, ldda) && K % 4 == 0;
  return status(launch_grouped(a, kDgrad, dtype == MOE_FP16, stream));
}

int moe_grouped_gemm_wgrad(int32_t dtype, const void *dC, int64_t lddc, const void *A, int64_t lda, int32_t a_rows,
                           const int32_t *a_row, const int32_t *offsets, int32_t G, int32_t P, int32_t N, int32_t K,
                           void *dW, int32_t dw_dtype, int32_t accumulate, hipStream_t stream) {
  const int st = check_groups(dtype, dw_dtype, offsets, G, P, N, K);
  if (st != MOE_OK) return st;
  if (a_rows < 0 || lddc < N || lda < K) return MOE_EINVAL;
  if (!dW || !typed(dW, dw_dtype)) return MOE_EINVAL;
  if (accumulate && dw_dtype != MOE_FP32) return MOE_EUNSUPPORTED;
  if (P > 0 && (!dC || (!A && a_rows > 0) || !typed(dC, dtype) || !typed(A, dtype) || !aligned(a_row, 4))) return MOE_EINVAL;
  if (P == 0 && accumulate) return MOE_OK;
  GroupedArgs a{};
  a.rows = static_cast<const uint16_t *>(A);
  a.ld_rows = lda;
  a.a_row = a_row;
  a.a_rows = a_rows;
  a.w = static_cast<const uint16_t *>(dC);
  a.ld_w = lddc;
  a.offsets = offsets;
  a.G = G; a.P = P; a.N = N; a.K = K;
  a.out = dW;
  a.ld_out = K;
  a.out_f32 = dw_dtype == MOE_FP32;
  a.accumulate = accumulate != 0;
  a.vec = units(dC, lddc, N) && units(A, lda, K);
  a.wide = wide_tiles(a, kWgrad);
  a.vec_out = runs(dW, dw_dtype, K) && K % 4 == 0;
  return status(launch_grouped(a, kWgrad, dtype == MOE_FP16, stream));
}

int moe_combine(int32_t dtype, const void *o, int64_t ldo, int32_t P, const int32_t *pair_pos, const float *w, int32_t T,
                int32_t k, int32_t d, const void *add, int32_t add_dtype, int64_t ldadd, void *y, int32_t y_dtype,
                int64_t ldy, hipStream_t stream) {
  if (!is16(dtype) || !out_type(y_dtype, dtype) || (add && !out_type(add_dtype, dtype))) return MOE_EINVAL;
  if (T < 0 || k < 1 || d < 1 || P < 0 || ldo < d || ldy < d || (add && ldadd < d)) return MOE_EINVAL;
  if (T > MOE_MAX_TOKENS || k > MOE_MAX_EXPERTS || d > kMaxExtent) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((P > 0 && !o) || !pair_pos || !y || !typed(o, dtype) || !typed(y, y_dtype) || !aligned(pair_pos, 4) || !aligned(w, 4)) return MOE_EINVAL;
  if (add && !typed(add, add_dtype)) return MOE_EINVAL;
  if (add == y && (add_dtype != y_dtype || (T > 1 && ldadd != ldy))) return MOE_EINVAL;
  CombineRowsArgs a{};
  a.o = static_cast<const uint16_t *>(o);
  a.ld_o = ldo;
  a.P = P;
  a.pos = pair_pos;
  a.w = w;
  a.T = T; a.k = k; a.d = d;
  a.add = add;
  a.add_f32 = add_dtype == MOE_FP32;
  a.ld_add = ldadd;
  a.y = y;
  a.y_f32 = y_dtype == MOE_FP32;
  a.ld_y = ldy;
  auto wide = [&](const void *p, int32_t t, int64_t ld) { return aligned(p, 16) && ld * size_of(t) % 16 == 0; };
  a.vec = d % 8 == 0 && wide(o, dtype, ldo) && wide(y, y_dtype, ldy) && (!add || wide(add, add_dtype, ldadd));
  return status(launch_combine_rows(a, dtype == MOE_FP16, stream));
}

int moe_combine_backward(int32_t dtype, const void *dy, int64_t lddy, const void *o, int64_t ldo, int32_t P,
                         const int32_t *pair_pos, const float *w, int32_t T, int32_t k, int32_t d, void *d_o,
                         int64_t lddo, float *dw, hipStream_t stream) {
  if (!is16(dtype) || T < 0 || k < 1 || d < 1 || P < 0 || lddy < d) return MOE_EINVAL;
  if ((d_o && lddo < d) || (dw && ldo < d) || (!d_o && !dw)) return MOE_EINVAL;
  if (T > MOE_MAX_TOKENS || k > MOE_MAX_EXPERTS || d > kMaxExtent) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dy || !pair_pos || !typed(dy, dtype) || !typed(d_o, dtype) || !aligned(pair_pos, 4) || !aligned(w, 4) || !aligned(dw, 4)) return MOE_EINVAL;
  if (dw && P > 0 && (!o || !typed(o, dtype))) return MOE_EINVAL;
  CombineRowsGradArgs a{};
  a.dy = static_cast<const uint16_t *>(dy);
  a.ld_dy = lddy;
  a.o = static_cast<const uint16_t *>(o);
  a.ld_o = ldo;
  a.P = P;
  a.pos = pair_pos;
  a.w = w;
  a.T = T; a.k = k; a.d = d;
  a.d_o = static_cast<uint16_t *>(d_o);
  a.ld_do = lddo;
  a.dw = dw;
  a.vec = units(dy, lddy, d) && (!dw || units(o, ldo, d)) && (!d_o || units(d_o, lddo, d));
  return status(launch_combine_rows_grad(a, dtype == MOE_FP16, stream));
}

int moe_adapter_plan(const int32_t *row_adapter, int32_t T, int32_t n, int32_t *rows, int32_t *offsets, hipStream_t stream) {
  if (T < 0 || n < 1 || !offsets || !aligned(offsets, 4)) return MOE_EINVAL;
  if (n > MOE_MAX_ADAPTERS || T > MOE_MAX_TOKENS) return MOE_EUNSUPPORTED;
  if (T > 0 && (!row_adapter || !rows || !aligned(row_adapter, 4) || !aligned(rows, 4))) return MOE_EINVAL;
  return status(launch_adapter_plan(row_adapter, T, n, rows, offsets, stream));
}

int moe_adapter_forward(int32_t dtype, const void *x, int64_t ldx, int32_t T, int32_t K, int32_t N, int32_t r, int32_t n,
                        const void *A, const void *B, const float *scale, const int32_t *rows, const int32_t *offsets,
                        const void *base, int64_t ldbase, void *y, int32_t y_dtype, int64_t ldy, hipStream_t stream) {
  const int st = check_adapter(dtype, static_cast<const uint16_t *>(x), ldx, T, K, N, r, n, static_cast<const uint16_t *>(A),
                               static_cast<const uint16_t *>(B), scale, rows, offsets);
  if (st != MOE_OK) return st;
  if (!out_type(y_dtype, dtype) || (base && ldbase < N) || ldy < N) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!y || !typed(y, y_dtype) || !typed(base, y_dtype) || (base == y && T > 1 && ldbase != ldy)) return MOE_EINVAL;
  AdapterArgs a{};
  a.x = static_cast<const uint16_t *>(x);
  a.ld_x = ldx;
  a.T = T; a.K = K; a.N = N; a.r = r; a.n = n;
  a.A = static_cast<const uint16_t *>(A);
  a.B = static_cast<const uint16_t *>(B);
  a.scale = scale;
  a.rows = rows;
  a.offsets = offsets;
  a.base = base;
  a.ld_base = ldbase;
  a.y = y;
  a.y_f32 = y_dtype == MOE_FP32;
  a.ld_y = ldy;
  a.vec_x = units(x, ldx, K) && units(A, K, K);
  auto wide = [&](const void *p, int64_t ld) { return aligned(p, 16) && ld * size_of(y_dtype) % 16 == 0; };
  a.vec_y = wide(y, ldy) && (!base || wide(base, ldbase));
  a.vec_b = units(B, r, r);
  return status(launch_adapter(a, dtype == MOE_FP16, stream));
}

size_t moe_adapter_backward_workspace_bytes(int32_t T, int32_t r) {
  if (T < 0 || r < 1 || T > MOE_MAX_TOKENS || r > MOE_MAX_ADAPTER_RANK) return 0;
  return (size_t)2 * (T ? T : 1) * 16 * rank_tiles(r) * sizeof(float);
}

int moe_adapter_backward(int32_t dtype, const void *dy, int64_t lddy, const void *x, int64_t ldx, int32_t T, int32_t K,
                         int32_t N, int32_t r, int32_t n, const void *A, const void *B, const float *scale,
                         const int32_t *rows, const int32_t *offsets, const void *dx_base, int64_t lddx_base, void *dx,
                         int32_t dx_dtype, int64_t lddx, void *dA, void *dB, int32_t g_dtype, int32_t accumulate, void *ws,
                         size_t ws_bytes, hipStream_t stream) {
  const int st = check_adapter(dtype, static_cast<const uint16_t *>(x), ldx, T, K, N, r, n, static_cast<const uint16_t *>(A),
                               static_cast<const uint16_t *>(B), scale, rows, offsets);
  if (st != MOE_OK) return st;
  if (!dx && !dA && !dB) return MOE_EINVAL;
  if (dx && (!out_type(dx_dtype, dtype) || lddx < K || (dx_base && lddx_base < K) || !typed(dx, dx_dtype) || !typed(dx_base, dx_dtype))) return MOE_EINVAL;
  if (dx && dx == dx_base && T > 1 && lddx != lddx_base) return MOE_EINVAL;
  if (lddy < N || (T > 0 && (!dy || !typed(dy, dtype)))) return MOE_EINVAL;
  if (dA || dB) {
    if (!out_type(g_dtype, dtype) || !typed(dA, g_dtype) || !typed(dB, g_dtype)) return MOE_EINVAL;
    if (accumulate && g_dtype != MOE_FP32) return MOE_EUNSUPPORTED;
    if (ws_bytes < moe_adapter_backward_workspace_bytes(T, r)) return MOE_EWORKSPACE;
    if (!ws || !aligned(ws, 256)) return MOE_EINVAL;
  }
  if (T == 0 && ((!dA && !dB) || accumulate)) return MOE_OK;
  AdapterGradArgs a{};
  a.dy = static_cast<const uint16_t *>(dy);
  a.x = static_cast<const uint16_t *>(x);
  a.ld_dy = lddy;
  a.ld_x = ldx;
  a.T = T; a.K = K; a.N = N; a.r = r; a.n = n;
  a.A = static_cast<const uint16_t *>(A);
  a.B = static_cast<const uint16_t *>(B);
  a.scale = scale;
  a.rows = rows;
  a.offsets = offsets;
  a.dx_base = dx_base;
  a.ld_dx_base = lddx_base;
  a.dx = dx;
  a.dx_f32 = dx_dtype == MOE_FP32;
  a.ld_dx = lddx;
  a.dA = dA;
  a.dB = dB;
  a.g_f32 = g_dtype == MOE_FP32;
  a.accumulate = accumulate != 0;
  if (dA || dB) {
    a.g = static_cast<float *>(ws);
    a.h = a.g + (size_t)T * 16 * rank_tiles(r);
  }
  a.vec_x = units(x, ldx, K) && units(A, K, K);
  a.vec_dy = units(dy, lddy, N);
  a.vec_b = units(B, r, r);
  auto wide = [&](const void *p, int64_t ld) { return aligned(p, 16) && ld * size_of(dx_dtype) % 16 == 0; };
  a.vec_da = runs(dA, g_dtype, 0) && K % 4 == 0;
  a.vec_dx = dx && wide(dx, lddx) && (!dx_base || wide(dx_base, lddx_base));
  return status(launch_adapter_grad(a, dtype == MOE_FP16, stream));
}

}  // extern "C"
