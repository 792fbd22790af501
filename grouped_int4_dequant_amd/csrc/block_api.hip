// C ABI of the operators of the block around the experts: argument validation
// and launches. Every check runs on the host before anything is enqueued; nothing here
// reads device memory, allocates or synchronises.

#include "api_checks.h"
#include "block_internal.h"

using namespace moe;

namespace {

constexpr int32_t kMaxFewWidth = 1 << 20;

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }
// A gradient's workspace: dz, then the chunks' column sums, then what the rows' parts give dW, then W and x in two bf16
// parts. Its size is that of the types that need most: dz in three parts, and fp16 operands.
int activation(int32_t act) { return act & ~MOE_ACT_ROUND_DZ; }
bool curved_act(int32_t act) { return activation(act) != MOE_ACT_NONE; }
int dz_parts(int32_t act) { return !curved_act(act) ? 0 : act & MOE_ACT_ROUND_DZ ? 1 : 3; }
size_t dz_part(int32_t T, int32_t N) { return pad256((size_t)T * N * 2); }
size_t dz_bytes(int32_t T, int32_t N, int32_t act) { return dz_parts(act) * dz_part(T, N); }
size_t halves_bytes(int32_t rows, int32_t K, int32_t act) { return dz_parts(act) > 1 ? 2 * pad256((size_t)rows * K * 2) : 0; }
// inner values of the few-token layer: fp32, in rows of whole 32-byte units
int32_t inner_pitch(int32_t f) { return (f + 7) / 8 * 8; }
size_t inner_bytes(int32_t rows, int32_t f) { return pad256((size_t)rows * inner_pitch(f) * sizeof(float)); }
size_t parts_bytes(const RowParts &p, int32_t N, int32_t K) { return p.count > 1 ? pad256((size_t)p.count * N * K * sizeof(float)) : 0; }
int64_t sums_pitch(int32_t n) { return ((int64_t)n + 7) / 8 * 8; }

size_t db_bytes(int32_t T, int32_t N, int32_t act) {
  act = activation(act);
  return pad256((size_t)column_chunks(T, is_gated(act) ? N / 2 : N).count * sums_pitch(N) * sizeof(float) + 1);
}

int check_linear(int32_t dtype, int32_t T, int32_t N, int32_t K, int32_t act) {
  if (!is16(dtype) || T < 0 || N < 1 || K < 1 || act < MOE_ACT_NONE || act > MOE_ACT_GEGLU) return MOE_EINVAL;
  if (is_gated(act) && N % 2 != 0) return MOE_EINVAL;
  if (T > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_layer16(const moe_layer16_t *L, int32_t T) {
  if (!L || !is16(L->dtype) || L->d < 1 || L->f < 1 || L->E < 1 || L->k < 1 || L->k > L->E || L->f_sh < 0 || T < 0) return MOE_EINVAL;
  if (L->E > MOE_MAX_EXPERTS || L->k > 64 || T > kFewTokens || T * L->k > kFewPairs) return MOE_EUNSUPPORTED;
  if (L->d > kMaxFewWidth || L->f > kMaxFewWidth || L->f_sh > kMaxFewWidth) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// One matrix as the tiles take it; rows: T of them.
void fill_dense(GroupedArgs &a, const void *rows, int64_t ld_rows, const void *w, int64_t ld_w, int32_t T, int32_t N, int32_t K) {
  a.rows = static_cast<const uint16_t *>(rows);
  a.ld_rows = ld_rows;
  a.a_rows = T;
  a.w = static_cast<const uint16_t *>(w);
  a.ld_w = ld_w;
  a.G = 1; a.P = T; a.N = N; a.K = K;
}
// An fp16 matrix that takes part as two bf16 parts at `to`.
HalvesArgs halves(const void *from, int64_t ld, int32_t rows, int32_t cols, char *to) {
  HalvesArgs h{};
  h.from = static_cast<const uint16_t *>(from);
  h.ld = ld;
  h.rows = rows;
  h.cols = cols;
  h.to = reinterpret_cast<uint16_t *>(to);
  h.next = (int64_t)pad256((size_t)rows * cols * 2) / 2;
  return h;
}

template <bool Gated>
int run_linear(int32_t dtype, const void *x, int64_t ldx, int32_t T, int32_t N, int32_t K, const void *W, const void *bias,
               int32_t bias_dtype, int32_t act, const void *residual, int64_t ldres, void *pre, int64_t ldpre, void *y,
               int32_t y_dtype, int64_t ldy, hipStream_t stream) {
  LinearArgs<Gated> a{};
  fill_dense(a, x, ldx, W, K, T, N, K);
  a.out = y;
  a.ld_out = ldy;
  a.out_f32 = y_dtype == MOE_FP32;
  a.vec = units(x, ldx, K) && units(W, K, K);
  a.wide = wide_tiles_dense(a, Gated);
  a.bias = bias;
  a.bias_f32 = bias_dtype == MOE_FP32;
  a.act = act;
  a.res = residual;
  a.ld_res = ldres;
  a.pre = static_cast<uint16_t *>(pre);
  a.ld_pre = ldpre;
  return status(launch_linear(a, dtype == MOE_FP16, stream));
}

}  // namespace

extern "C" {

int moe_linear(int32_t dtype, const void *x, int64_t ldx, int32_t T, int32_t N, int32_t K, const void *W, const void *bias,
               int32_t bias_dtype, int32_t act, const void *residual, int64_t ldres, void *pre, int64_t ldpre, void *y,
               int32_t y_dtype, int64_t ldy, hipStream_t stream) {
  const int st = check_linear(dtype, T, N, K, act);
  if (st != MOE_OK) return st;
  const int32_t cols = is_gated(act) ? N / 2 : N;
  if (!out_type(y_dtype, dtype) || (bias && !out_type(bias_dtype, dtype))) return MOE_EINVAL;
  if (ldx < K || ldy < cols || (residual && ldres < cols) || (pre && ldpre < N)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!x || !W || !y || !typed(x, dtype) || !typed(W, dtype) || !typed(y, y_dtype) || !typed(residual, y_dtype) || !typed(pre, dtype)) return MOE_EINVAL;
  if ((bias && !typed(bias, bias_dtype)) || (residual == y && T > 1 && ldres != ldy)) return MOE_EINVAL;
  return is_gated(act) ? run_linear<true>(dtype, x, ldx, T, N, K, W, bias, bias_dtype, act, residual, ldres, pre, ldpre, y, y_dtype, ldy, stream)
                       : run_linear<false>(dtype, x, ldx, T, N, K, W, bias, bias_dtype, act, residual, ldres, pre, ldpre, y, y_dtype, ldy, stream);
}

size_t moe_linear_backward_workspace_bytes(int32_t T, int32_t N, int32_t K, int32_t act) {
  if (check_linear(MOE_BF16, T, N, K, activation(act)) != MOE_OK) return 0;
  const size_t wide = parts_bytes(weight_parts(T, N, K, true), N, K), small = parts_bytes(weight_parts(T, N, K, false), N, K);
  return dz_bytes(T, N, act) + db_bytes(T, N, act) + (wide > small ? wide : small) + halves_bytes(N, K, act) + halves_bytes(T, K, act);
}

int moe_linear_backward(int32_t dtype, const void *dy, int64_t lddy, const void *x, int64_t ldx, int32_t T, int32_t N, int32_t K,
                        const void *W, const void *pre, int64_t ldpre, int32_t act_flags, void *dx, int32_t dx_dtype, int64_t lddx,
                        void *dW, void *db, int32_t g_dtype, int32_t accumulate, void *ws, size_t ws_bytes, hipStream_t stream) {
  const int32_t act = activation(act_flags);
  const int st = check_linear(dtype, T, N, K, act);
  if (st != MOE_OK) return st;
  const int32_t cols = is_gated(act) ? N / 2 : N;
  const bool curved = act != MOE_ACT_NONE;
  if (T > 0 && !dx && !dW && !db) return MOE_EINVAL;
  if (lddy < cols || (curved && ldpre < N)) return MOE_EINVAL;
  if (dx && (!out_type(dx_dtype, dtype) || lddx < K || !typed(dx, dx_dtype))) return MOE_EINVAL;
  if ((dW || db) && (!out_type(g_dtype, dtype) || !typed(dW, g_dtype) || !typed(db, g_dtype))) return MOE_EINVAL;
  if (dW && ldx < K) return MOE_EINVAL;
  if ((dW || db) && accumulate && g_dtype != MOE_FP32) return MOE_EUNSUPPORTED;
  if (T > 0) {
    if (!dy || !typed(dy, dtype) || (curved && (!pre || !typed(pre, dtype)))) return MOE_EINVAL;
    if ((dx && (!W || !typed(W, dtype))) || (dW && (!x || !typed(x, dtype)))) return MOE_EINVAL;
  }
  if (curved || db || dW) {
    if (ws_bytes < moe_linear_backward_workspace_bytes(T, N, K, act_flags)) return MOE_EWORKSPACE;
    if (!ws || !aligned(ws, 256)) return MOE_EINVAL;
  }
  if (T == 0 && ((!dW && !db) || accumulate)) return MOE_OK;
  const bool fp16 = dtype == MOE_FP16;
  // An fp32 result takes dz whole, in three bf16 parts, a 16-bit one in two. fp16's exponents hold no such
  // parts: where one of the results is fp32, fp16 operands take part as two bf16 parts each.
  const bool dx_f32 = dx && dx_dtype == MOE_FP32, dW_f32 = dW && g_dtype == MOE_FP32;
  const bool split = curved && !(act_flags & MOE_ACT_ROUND_DZ), whole = dx_f32 || dW_f32, bf16_parts = split && fp16 && whole;
  const void *dz = dy;
  int64_t lddz = lddy;
  ActGradArgs c{};
  c.dy = static_cast<const uint16_t *>(dy);
  c.ld_dy = lddy;
  c.pre = static_cast<const uint16_t *>(pre);
  c.ld_pre = ldpre;
  c.T = T; c.N = N; c.cols = cols; c.act = act;
  const ColumnChunks n = column_chunks(T, cols);
  c.chunk_rows = n.rows;
  c.chunks = T > 0 ? n.count : 0;
  if (curved) {
    c.dz = static_cast<uint16_t *>(ws);
    c.dz_parts = !split ? 1 : whole ? 3 : 2;
    c.dz_next = (int64_t)dz_part(T, N) / 2;
    dz = ws;
    lddz = N;
  }
  if (db) {
    c.part = reinterpret_cast<float *>(static_cast<char *>(ws) + dz_bytes(T, N, act_flags));
    c.pitch = sums_pitch(N);
    c.db = db;
    c.g_f32 = g_dtype == MOE_FP32;
    c.accumulate = accumulate != 0;
  }
  const RowParts wide_rows = weight_parts(T, N, K, true), small_rows = weight_parts(T, N, K, false);
  char *const parts = static_cast<char *>(ws) + dz_bytes(T, N, act_flags) + db_bytes(T, N, act_flags);
  const size_t wide_bytes = parts_bytes(wide_rows, N, K), small_bytes = parts_bytes(small_rows, N, K);
  HalvesArgs w2{}, x2{};
  if (bf16_parts) {
    char *const at = parts + (wide_bytes > small_bytes ? wide_bytes : small_bytes);
    if (dx && T > 0) {
      w2 = halves(W, K, N, K, at);
      W = w2.to;
    }
    if (dW) {
      x2 = halves(x, ldx, T, K, at + halves_bytes(N, K, act_flags));
      x = x2.to;
      ldx = K;
    }
  }
  SplitArgs dxa{}, dwa{};
  if (dx) {
    fill_dense(dxa, dz, lddz, W, K, T, N, K);
    dxa.out = dx;
    dxa.ld_out = lddx;
    dxa.out_f32 = dx_dtype == MOE_FP32;
    dxa.vec = units(dz, lddz, N) && units(W, K, K);
    dxa.wide = wide_tiles_dense(dxa, false);
    dxa.vec_out = runs(dx, dx_dtype, lddx) && K % 4 == 0;
    dxa.c_parts = dx_f32 ? 3 : 2;
    dxa.o_parts = bf16_parts ? 2 : 1;
    dxa.c_next = c.dz_next;
    dxa.o_next = w2.next;
  }
  if (dW) {
    fill_dense(dwa, x, ldx, dz, lddz, T, N, K);
    dwa.out = dW;
    dwa.ld_out = K;
    dwa.out_f32 = g_dtype == MOE_FP32;
    dwa.accumulate = accumulate != 0;
    dwa.vec = units(dz, lddz, N) && units(x, ldx, K);
    dwa.wide = wide_tiles_dense(dwa, false);
    const RowParts &p = dwa.wide ? wide_rows : small_rows;
    dwa.part_rows = p.rows;
    dwa.G = p.count;
    dwa.vec_out = runs(dW, g_dtype, K) && K % 4 == 0;
    dwa.c_parts = dW_f32 ? 3 : 2;
    dwa.o_parts = bf16_parts ? 2 : 1;
    dwa.c_next = c.dz_next;
    dwa.o_next = x2.next;
  }
  float *const sums = reinterpret_cast<float *>(parts);
  return status(split ? launch_linear_grad_split(c, dxa, dwa, w2, x2, sums, fp16, bf16_parts, stream) : launch_linear_grad(c, dxa, dwa, sums, fp16, stream));
}

int moe_residual_norm(int32_t dtype, const void *o, int64_t ldo, const void *x, int64_t ldx, int32_t stream_dtype, int32_t T,
                      int32_t d, const void *w_o, const void *gate, int32_t gates, const void *w_n, int32_t w_dtype, float scale,
                      float eps, void *y, int64_t ldy, void *n, int64_t ldn, hipStream_t stream) {
  if (!is16(dtype) || !out_type(stream_dtype, dtype) || T < 0 || d < 1 || !(eps >= 0.f)) return MOE_EINVAL;
  if (!o) w_o = gate = nullptr;
  if (!n) w_n = nullptr;
  if ((w_o || gate || w_n) && !out_type(w_dtype, dtype)) return MOE_EINVAL;
  if ((n && !w_n) || (gate && (gates < 1 || T % gates != 0))) return MOE_EINVAL;
  if ((o && ldo < d) || (x && ldx < d) || (y && ldy < d) || (n && ldn < d)) return MOE_EINVAL;
  if (d > MOE_MAX_NORM_WIDTH || T > kMaxExtent) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((!o && !x) || (!y && !n) || !typed(o, dtype) || !typed(x, stream_dtype) || !typed(y, stream_dtype) || !typed(n, dtype)) return MOE_EINVAL;
  if (!typed(w_o, w_dtype) || !typed(gate, w_dtype) || !typed(w_n, w_dtype)) return MOE_EINVAL;
  if (T > 1 && ((y && y == x && ldy != ldx) || (n && n == o && ldn != ldo))) return MOE_EINVAL;
  NormArgs a{};
  a.o = static_cast<const uint16_t *>(o);
  a.ld_o = ldo;
  a.x = x;
  a.ld_x = ldx;
  a.w_o = w_o; a.gate = gate; a.w_n = w_n;
  a.w_f32 = w_dtype == MOE_FP32;
  a.stream_f32 = stream_dtype == MOE_FP32;
  a.period = gate ? T / gates : T;
  a.T = T; a.d = d; a.scale = scale; a.eps = eps;
  a.y = y;
  a.ld_y = ldy;
  a.n = static_cast<uint16_t *>(n);
  a.ld_n = ldn;
  return status(launch_norm(a, dtype == MOE_FP16, stream));
}

size_t moe_residual_norm_backward_workspace_bytes(int32_t T, int32_t d, int32_t gates) {
  if (T < 0 || d < 1 || gates < 1 || T % gates != 0 || d > MOE_MAX_NORM_WIDTH || T > kMaxExtent) return 0;
  const NormChunks c = norm_chunks(T, T > 0 ? T / gates : 1);
  return pad256((size_t)3 * (c.count > 0 ? c.count : 1) * sums_pitch(d) * sizeof(float));
}

int moe_residual_norm_backward(int32_t dtype, const void *dy, int64_t lddy, const void *dn, int64_t lddn, const void *o, int64_t ldo,
                               const void *y, int64_t ldy, int32_t stream_dtype, int32_t T, int32_t d, const void *w_o,
                               const void *gate, int32_t gates, const void *w_n, int32_t w_dtype, float scale, float eps, void *dx,
                               int64_t lddx, void *d_o, int64_t lddo, void *dw_o, void *dgate, void *dw_n, int32_t g_dtype,
                               int32_t accumulate, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (!is16(dtype) || !out_type(stream_dtype, dtype) || T < 0 || d < 1 || !(eps >= 0.f)) return MOE_EINVAL;
  // What is formed from what: a T of zero has no rows whose pointers would tell, so the weights do.
  if (!gate) gates = 1;
  if (gates < 1 || T % gates != 0) return MOE_EINVAL;
  const bool sums = dw_o || dgate || dw_n;
  if ((T > 0 && !dx && !d_o && !sums) || (dw_o && !w_o) || (dgate && !gate) || (dw_n && !w_n)) return MOE_EINVAL;
  if ((w_o || gate || w_n) && !out_type(w_dtype, dtype)) return MOE_EINVAL;
  if (sums && (!out_type(g_dtype, dtype) || !typed(dw_o, g_dtype) || !typed(dgate, g_dtype) || !typed(dw_n, g_dtype))) return MOE_EINVAL;
  if ((dy && lddy < d) || (dn && (lddn < d || ldy < d)) || (o && ldo < d) || (dx && lddx < d) || (d_o && lddo < d)) return MOE_EINVAL;
  if (d > MOE_MAX_NORM_WIDTH || T > kMaxExtent || (sums && accumulate && g_dtype != MOE_FP32)) return MOE_EUNSUPPORTED;
  if (sums) {
    if (ws_bytes < moe_residual_norm_backward_workspace_bytes(T, d, gates)) return MOE_EWORKSPACE;
    if (!ws || !aligned(ws, 256)) return MOE_EINVAL;
  }
  if (T == 0 && (!sums || accumulate)) return MOE_OK;
  if (T > 0) {
    if ((!dy && !dn) || (dn && (!w_n || !y)) || ((d_o || dw_o || dgate) && !o) || (dw_n && !dn)) return MOE_EINVAL;
    if (!typed(dy, stream_dtype) || !typed(dn, dtype) || !typed(o, dtype) || !typed(y, stream_dtype) || !typed(dx, stream_dtype) || !typed(d_o, dtype)) return MOE_EINVAL;
    if (!typed(w_o, w_dtype) || !typed(gate, w_dtype) || !typed(w_n, w_dtype)) return MOE_EINVAL;
    if (T > 1 && dx && dx == dy && lddx != lddy) return MOE_EINVAL;
  }
  const bool block = o && (d_o || dw_o || dgate);
  NormGradArgs a{};
  a.dy = dy;
  a.ld_dy = lddy;
  a.dn = static_cast<const uint16_t *>(dn);
  a.ld_dn = lddn;
  a.o = block ? static_cast<const uint16_t *>(o) : nullptr;
  a.ld_o = ldo;
  a.y = y;
  a.ld_y = ldy;
  a.w_o = block ? w_o : nullptr;
  a.gate = block ? gate : nullptr;
  a.w_n = w_n;
  a.w_f32 = w_dtype == MOE_FP32;
  a.stream_f32 = stream_dtype == MOE_FP32;
  a.gates = gates;
  a.period = T > 0 ? T / gates : 1;
  a.T = T; a.d = d; a.scale = scale; a.eps = eps;
  a.dx = dx;
  a.ld_dx = lddx;
  a.d_o = static_cast<uint16_t *>(d_o);
  a.ld_do = lddo;
  a.dw_o = dw_o; a.dgate = dgate; a.dw_n = dw_n;
  a.g_f32 = g_dtype == MOE_FP32;
  a.accumulate = accumulate != 0;
  a.part = static_cast<float *>(ws);
  a.pitch = sums_pitch(d);
  const NormChunks c = norm_chunks(T, a.period);
  a.chunk_rows = c.rows;
  a.chunks = T > 0 ? c.count : 0;
  a.per_gate = c.per_gate;
  if (T == 0) a.per_gate = 0;
  return status(launch_norm_grad(a, dtype == MOE_FP16, stream));
}

size_t moe_few_tokens_workspace_bytes(const moe_layer16_t *L, int32_t T) {
  if (check_layer16(L, T) != MOE_OK) return 0;
  return pad256(sizeof(FewPlan)) + inner_bytes(T * L->k, L->f) + inner_bytes(T, L->f_sh);
}

int moe_few_tokens_layer(const moe_layer16_t *L, const void *x, int64_t ldx, const float *logits, int32_t T, const void *add,
                         int64_t ldadd, void *y, int32_t y_dtype, int64_t ldy, int32_t *topk_ids, float *topk_w, void *ws,
                         size_t ws_bytes, hipStream_t stream) {
  const int st = check_layer16(L, T);
  if (st != MOE_OK) return st;
  if (!out_type(y_dtype, L->dtype) || ldx < L->d || ldy < L->d || (add && ldadd < L->d)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!x || !logits || !y || !L->gu || !L->dn || !typed(x, L->dtype) || !aligned(logits, 4) || !typed(y, y_dtype)) return MOE_EINVAL;
  if (!typed(L->gu, L->dtype) || !typed(L->dn, L->dtype) || !typed(add, y_dtype) || !aligned(topk_ids, 4) || !aligned(topk_w, 4)) return MOE_EINVAL;
  if (L->f_sh > 0 && (!L->sh_gu || !L->sh_dn || !typed(L->sh_gu, L->dtype) || !typed(L->sh_dn, L->dtype))) return MOE_EINVAL;
  if (add == y && T > 1 && ldadd != ldy) return MOE_EINVAL;
  if (ws_bytes < moe_few_tokens_workspace_bytes(L, T)) return MOE_EWORKSPACE;
  if (!ws || !aligned(ws, 256)) return MOE_EINVAL;
  FewArgs a{};
  a.x = static_cast<const uint16_t *>(x);
  a.ld_x = ldx;
  a.logits = logits;
  a.T = T; a.d = L->d; a.f = L->f; a.f_sh = L->f_sh; a.E = L->E; a.k = L->k;
  a.gu = static_cast<const uint16_t *>(L->gu);
  a.dn = static_cast<const uint16_t *>(L->dn);
  a.sh_gu = static_cast<const uint16_t *>(L->sh_gu);
  a.sh_dn = static_cast<const uint16_t *>(L->sh_dn);
  a.add = add;
  a.ld_add = ldadd;
  a.y = y;
  a.y_f32 = y_dtype == MOE_FP32;
  a.ld_y = ldy;
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  char *p = static_cast<char *>(ws);
  a.plan = reinterpret_cast<FewPlan *>(p);
  a.h = reinterpret_cast<float *>(p + pad256(sizeof(FewPlan)));
  a.h_sh = reinterpret_cast<float *>(p + pad256(sizeof(FewPlan)) + inner_bytes(T * L->k, L->f));
  a.pitch = inner_pitch(L->f);
  a.pitch_sh = inner_pitch(L->f_sh);
  return status(launch_few_layer(a, L->dtype == MOE_FP16, stream));
}

}  // extern "C"
