// The matrix product with bias, activation and residual, and its gradients, for
// gfx950.
//
//   z = x W^T + b     y = act(z) + r       act(z) = curve(z), or curve(z[:f]) z[f:] if gated (N = 2 f)
//   dz = act'(z) dy   dx = dz W   dW = dz^T x   db = sum_t dz
//
// Many rows are bound by the matrix instructions and take the tiles of grouped_tiles.h,
// with the epilogue on the accumulators: z, the activation and the residual never make a trip
// of their own. Few rows are bound by reading W once.
// bf16: 8192 rows, 8192 x 2048, swiglu with z stored 243 us on inputs in cache (1130 TFLOP/s; the product alone 218, a
// library's 203), 265 from memory; 1 row, 4096 x 2048 5.9 us.
// dz is an operand of its two products, which have 16 bits a value, and is laid out as a sum of such: rounded to one, it
// makes 16-bit results 1.4 times as far off as their own rounding (bf16 2.35e-3 against 1.66e-3) and fp32 ones 2800 times. Two parts for
// 16-bit results and three for fp32 ones cost as many products: 4096 rows, 8192 x 2048, bf16, each product 115 us a part.

#include "grouped_tiles.h"
#include "block_internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- few rows
// At most 64 rows: a workgroup takes 16 rows of W (gated: eight of the gate and the eight that
// it multiplies), whose sums its eight waves share and join in LDS, in order. W goes straight
// from memory to operand registers and is read once; x comes from L2. 4096 x 2048, bf16: 1 row 5.9 us, 16 rows 7.2,
// 64 rows 12.9.
template <typename Tr, bool Gated, int RB>
__global__ __launch_bounds__(512) void linear_few_kernel(LinearArgs<Gated> a) {
  constexpr int kDeep = 8, kXDeep = RB == 1 ? 8 : RB == 2 ? 4 : 2;  // requests of W, and of each row block of x, in flight
  __shared__ __attribute__((aligned(16))) f4 s_part[8][RB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;
  constexpr int C = Gated ? 8 : 16;  // result columns
  const int J = Gated ? a.N / 2 : a.N, j0 = blockIdx.x * C;
  const int col = Gated ? j0 + (p16 & 7) : j0 + p16;
  const uint16_t *w = col < J ? a.w + (int64_t)(Gated && p16 >= 8 ? J + col : col) * a.K : nullptr;
  const uint16_t *x[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) x[b] = 16 * b + p16 < a.P ? a.rows + (int64_t)(16 * b + p16) * a.ld_rows : nullptr;
  const s8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  f4 acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f4{0.f, 0.f, 0.f, 0.f};
  // the wave that joins a block of rows: lane has row p16, W's rows 4 q4 ..
  const int row = 16 * wave + p16, c = j0 + 4 * q4;
  const bool mine = wave < RB && row < a.P && c < J && (!Gated || q4 < 2);
  Extra4 extra;
  if (mine) extra = extra4<Tr>(a, row, c, J - c);
  for (int k0 = 32 * wave; k0 < a.K; k0 += 256 * kDeep) {
    s8 wv[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int k = k0 + 256 * u + 8 * q4;
      wv[u] = w && k < a.K ? *reinterpret_cast<const s8 *>(w + k) : zero;
    }
#pragma unroll
    for (int u0 = 0; u0 < kDeep; u0 += kXDeep) {
      s8 xv[kXDeep][RB];
#pragma unroll
      for (int u = 0; u < kXDeep; ++u)
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const int k = k0 + 256 * (u0 + u) + 8 * q4;
          xv[u][b] = x[b] && k < a.K ? *reinterpret_cast<const s8 *>(x[b] + k) : zero;
        }
#pragma unroll
      for (int u = 0; u < kXDeep; ++u)
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b] = Tr::mfma(wv[u0 + u], xv[u][b], acc[b]);
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b) s_part[wave][b][lane] = acc[b];
  __syncthreads();
  if (wave >= RB) return;
  f4 v = s_part[0][wave][lane];
#pragma unroll
  for (int y = 1; y < 8; ++y) v += s_part[y][wave][lane];
  f4 u = v;
  if constexpr (Gated) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __shfl(v[i], (lane + 32) & 63);
  }
  if (mine) finish4<Tr>(a, row, c, min(J - c, 4), v, u, extra);
}

// ------------------------------------------------------- activation's gradient
// Operands in fp16 whose products are formed of bf16 parts, which have fp32's exponents.
struct Fp16InBf16 : Fp16 {
  static __device__ __forceinline__ f4 mfma(s8 a, s8 b, f4 c) { return Bf16::mfma(a, b, c); }
};
template <typename Tr>
struct PartOf { typedef Tr type; };
template <>
struct PartOf<Fp16InBf16> { typedef Bf16 type; };

// The value of a 16-bit type next to a finite v, towards zero.
template <typename P>
__device__ __forceinline__ uint16_t towards_zero(float v) {
  if constexpr (std::is_same<P, Bf16>::value) return (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16);
  else return (uint16_t)__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(fminf(fmaxf(v, -65504.f), 65504.f), 0.f));
}
// v as the sum of `n` (2 or 3, bf16) parts. All are of v's sign, and none is zero unless v is (or is less than two of the type's smallest
// steps): the product of each with an infinite value is then the infinity that v's is, and the sum of the products too. So a value
// that its first part would hold whole takes the next smaller one there. The last of two parts is rounded, the last of three exact.
template <typename P, int N>
__device__ __forceinline__ void split(float v, uint16_t (&part)[N]) {
  if (!(__builtin_fabsf(v) < __builtin_inff())) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[i] = P::from(v);
    return;
  }
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) {
    uint16_t p = towards_zero<P>(v);
    float rest = v - P::to(p);
    if ((i + 2 < N ? rest == 0.f : (P::from(rest) & 0x7fff) == 0) && (p & 0x7fff) > 1) {
      --p;  // one step towards zero, whatever the sign
      rest = v - P::to(p);
    }
    part[i] = p;
    v = rest;
  }
  part[N - 1] = P::from(v);
}
// The same of eight values, and their first `left` stored: [N][next]
template <typename P, int N>
__device__ __forceinline__ void store_parts(uint16_t *to, int64_t at, int64_t next, int left, const float (&v)[8]) {
  uint16_t part[8][N];
#pragma unroll
  for (int i = 0; i < 8; ++i) split<P, N>(v[i], part[i]);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint16_t *q = to + n * next + at;
    if (left >= 8) {
      u4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)part[2 * i][n] | (uint32_t)part[2 * i + 1][n] << 16;
      *reinterpret_cast<u4_elem *>(q) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = part[i][n];
    }
  }
}

// An fp16 matrix as two bf16 parts, exactly. Eight elements a thread; bound by memory.
__global__ __launch_bounds__(256) void halves_kernel(HalvesArgs a) {
  const int units = (a.cols + 7) / 8;
  const int64_t all = (int64_t)a.rows * units;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < all; u += (int64_t)gridDim.x * 256) {
    const int64_t row = u / units;
    const int col = 8 * (int)(u - row * units), left = a.cols - col;
    float v[8];
    widen8<Fp16, false>(load_raw8<false>(a.from, row * a.ld + col, left), v);
    store_parts<Bf16, 2>(a.to, row * a.cols + col, a.next, left, v);
  }
}

// A workgroup takes 256 columns of a chunk of rows; a thread eight of them, every eighth row. dz enters the two products
// as an operand of the matrix instructions, in 16-bit parts; the column sums are of its values before
// that. Bound by memory: 4096 x 8192, swiglu, 37 us for 168 MB where dz is rounded (45 with db), 55 for 235 MB in two parts.
template <typename Tr, bool Gated>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  __shared__ float s_sum[8][Gated ? 2 : 1][256];
  const int unit = threadIdx.x & 31, r0 = threadIdx.x >> 5;
  const int col = 256 * blockIdx.x + 8 * unit, left = a.cols - col;
  const int begin = blockIdx.y * a.chunk_rows, end = min(begin + a.chunk_rows, a.T);
  float sum[Gated ? 2 : 1][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sum[0][i] = 0.f;
    if constexpr (Gated) sum[1][i] = 0.f;
  }
  if (left > 0) {
    Raw8 dyv, zv, uv;
    auto load = [&](int row) __attribute__((always_inline)) {
      const int n = row < end ? left : 0;
      dyv = load_raw8<false>(a.dy, (int64_t)row * a.ld_dy + col, n);
      if (a.act == MOE_ACT_NONE) return;
      zv = load_raw8<false>(a.pre, (int64_t)row * a.ld_pre + col, n);
      if constexpr (Gated) uv = load_raw8<false>(a.pre, (int64_t)row * a.ld_pre + a.cols + col, n);
    };
    load(begin + r0);
    for (int row = begin + r0; row < end; row += 8) {
      float dy[8], z[8], u[8];
      widen8<Tr, false>(dyv, dy);
      if (a.act != MOE_ACT_NONE) {
        widen8<Tr, false>(zv, z);
        if constexpr (Gated) widen8<Tr, false>(uv, u);
      }
      load(row + 8);
      if (a.act != MOE_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float value;
          const float slope = slope_of(a.act, z[i], value);
          if constexpr (Gated) {
            z[i] = dy[i] * value;
            dy[i] = dy[i] * u[i] * slope;
          } else {
            dy[i] *= slope;
          }
        }
        auto store = [&](int64_t at, const float (&v)[8]) __attribute__((always_inline)) {
          typedef typename PartOf<Tr>::type P;
          if (a.dz_parts == 1) store8<Tr>(a.dz, false, at, left, v);
          else if (std::is_same<P, Bf16>::value && a.dz_parts == 3) store_parts<P, std::is_same<P, Bf16>::value ? 3 : 2>(a.dz, at, a.dz_next, left, v);
          else store_parts<P, 2>(a.dz, at, a.dz_next, left, v);
        };
        store((int64_t)row * a.N + col, dy);
        if constexpr (Gated) store((int64_t)row * a.N + a.cols + col, z);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0][i] += dy[i];
        if constexpr (Gated) sum[1][i] += z[i];
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s_sum[r0][0][8 * unit + i] = sum[0][i];
    if constexpr (Gated) s_sum[r0][1][8 * unit + i] = sum[1][i];
  }
  __syncthreads();
  const int c = 256 * blockIdx.x + threadIdx.x;
  if (c >= a.cols) return;
#pragma unroll
  for (int h = 0; h < (Gated ? 2 : 1); ++h) {
    float f = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) f += s_sum[r][h][threadIdx.x];
    a.part[(int64_t)blockIdx.y * a.pitch + h * a.cols + c] = f;
  }
}

template <typename Tr>
__device__ __forceinline__ void store_db(const ActGradArgs &a, int col, float f) {
  if (a.g_f32) {
    float *q = static_cast<float *>(a.db) + col;
    *q = a.accumulate ? *q + f : f;
  } else {
    static_cast<uint16_t *>(a.db)[col] = Tr::from(f);
  }
}

// db: the chunks' column sums added up in order. 64 columns a workgroup, its waves share the chunks.
template <typename Tr, int Waves>
__device__ __forceinline__ void add_chunks(const ActGradArgs &a, int block, float *s_part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = block * 64 + lane;
  float f = 0.f;
  if (col < a.N) {
    for (int c = wave; c < a.chunks; c += 8 * Waves) {
      float v[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        v[y] = 0.f;
        if (c + Waves * y < a.chunks) v[y] = a.part[(int64_t)(c + Waves * y) * a.pitch + col];
      }
#pragma unroll
      for (int y = 0; y < 8; ++y) f += v[y];
    }
  }
  s_part[64 * wave + lane] = f;
  __syncthreads();
  if (wave != 0 || col >= a.N) return;
  f = 0.f;
#pragma unroll
  for (int w = 0; w < Waves; ++w) f += s_part[64 * w + lane];
  store_db<Tr>(a, col, f);
}
template <typename Tr>
__global__ __launch_bounds__(1024) void column_sums_kernel(ActGradArgs a) {
  __shared__ float s_part[1024];
  add_chunks<Tr, 16>(a, blockIdx.x, s_part);
}

// db without activation, of few rows: 64 columns a workgroup, eight a thread, every 32nd row.
template <typename Tr>
__device__ __forceinline__ void add_rows(const ActGradArgs &a, int block, float *s_part) {
  const int unit = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int col = 64 * block + 8 * unit, left = a.N - col;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int row = r0; row < a.T; row += 128) {
    Raw8 v[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = load_raw8<false>(a.dy, (int64_t)(row + 32 * y) * a.ld_dy + col, row + 32 * y < a.T ? left : 0);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float f[8];
      widen8<Tr, false>(v[y], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += f[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s_part[64 * r0 + 8 * unit + i] = sum[i];
  __syncthreads();
  const int c = 64 * block + threadIdx.x;
  if (threadIdx.x >= 64 || c >= a.N) return;
  float f = 0.f;
#pragma unroll
  for (int r = 0; r < 32; ++r) f += s_part[64 * r + threadIdx.x];
  store_db<Tr>(a, c, f);
}

// Both products and db of a gradient whose tiles are few, side by side in one launch: workgroups 0 .. n_w - 1 take
// dW's tiles, n_d more those of dx, the rest 64 columns of db each. 777 rows, 1032 x 520:
// 15 us, 30 in four launches.
template <typename Tr, bool Vec, typename Args>
__global__ __launch_bounds__(256) void linear_grad_small_kernel(Args dg, Args wg, ActGradArgs c, bool rows, int n_w, int n_d) {
  __shared__ __attribute__((aligned(16))) SmallTile s_l[2], s_r[2];
  const int b = blockIdx.x;
  if (b < n_w) {
    small_body<Tr, kWgrad, Vec, 4>(wg, b, s_l, s_r);
  } else if (b < n_w + n_d) {
    small_body<Tr, kDgrad, Vec, 4>(dg, b - n_w, s_l, s_r);
  } else {
    float *part = reinterpret_cast<float *>(s_l);
    if (rows) add_rows<Tr>(c, b - n_w - n_d, part);
    else add_chunks<Tr, 4>(c, b - n_w - n_d, part);
  }
}

// dW out of the parts' sums, in order. Four elements a thread; bound by memory.
template <typename Tr>
__global__ __launch_bounds__(256) void add_parts_kernel(const float *parts, int32_t count, int64_t n, void *out, bool f32, bool accumulate) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  const int left = (int)min(n - at, (int64_t)4);
  f4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < count; p += 4) {
    f4 v[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = load4<Tr>(parts, true, (int64_t)min(p + y, count - 1) * n + at, left);
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (p + y < count) sum += v[y];
  }
  if (accumulate) sum += load4<Tr>(out, true, at, left);
  store4_of<Tr>(out, f32, at, left, sum);
}

template <typename Tr, bool Gated>
hipError_t linear_of(const LinearArgs<Gated> &a, hipStream_t s) {
  if (a.vec && a.P <= 64) {
    const int64_t wgs = cdiv(Gated ? a.N / 2 : a.N, Gated ? 8 : 16);
    if (!grid_fits(wgs, 512)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)wgs);
    if (a.P <= 16) linear_few_kernel<Tr, Gated, 1><<<grid, 512, 0, s>>>(a);
    else if (a.P <= 32) linear_few_kernel<Tr, Gated, 2><<<grid, 512, 0, s>>>(a);
    else linear_few_kernel<Tr, Gated, 4><<<grid, 512, 0, s>>>(a);
    return hipGetLastError();
  }
  return launch_vec<Tr, kFwd, LinearArgs<Gated>>(a, s);
}

template <typename Tr>
hipError_t act_grad_of(const ActGradArgs &a, bool add, hipStream_t s) {
  if (a.chunks > 0) {
    const dim3 grid((unsigned)cdiv(a.cols, 256), (unsigned)a.chunks);
    if (a.cols != a.N) act_grad_kernel<Tr, true><<<grid, 256, 0, s>>>(a);
    else act_grad_kernel<Tr, false><<<grid, 256, 0, s>>>(a);
  }
  if (add) column_sums_kernel<Tr><<<dim3((unsigned)cdiv(a.N, 64)), 1024, 0, s>>>(a);
  return hipGetLastError();
}

// Whether every form that the products of a gradient may take fits a launch: known before the first of a call's
// kernels is enqueued.
bool grad_fits(const ActGradArgs &c, const DenseArgs &dx, const DenseArgs &dw) {
  const int64_t n_w = dw.out ? dw.G * cdiv(dw.N, kSmall) * cdiv(dw.K, kSmall) : 0, n_d = dx.out ? xcd_grid(cdiv(c.T, kSmall) * cdiv(dx.K, kSmall)) : 0;
  const int64_t few = dx.out && c.T <= 64 ? cdiv(c.T, kFewRows) * cdiv(dx.K, 64) : 0;
  return grid_fits(n_w + n_d + cdiv(c.N, 64), 256) && grid_fits(few, 512) && grid_fits(c.db ? cdiv(c.N, 64) : 0, 1024) &&
         n_w + n_d + cdiv(c.N, 64) < INT32_MAX / 2;
}

template <typename Tr, typename Args>
hipError_t linear_grad_of(const ActGradArgs &c, const Args &dx, const Args &dw, float *parts, hipStream_t s) {
  const bool curved = c.act != MOE_ACT_NONE;
  // dW's tiles leave their sums in dW, or in the parts
  Args w = dw;
  const bool cut = dw.out && dw.G > 1;
  if (cut) {
    w.out = parts;
    w.out_f32 = 1;
    w.accumulate = 0;
    w.vec_out = dw.K % 4 == 0;
  }
  // one launch for what may run side by side, where both products take small tiles
  const bool small = dx.out && dw.out && c.T > 0 && dense_tile_rows<kDgrad>(dx) == kSmall && dense_tile_rows<kWgrad>(w) == kSmall && dx.vec == dw.vec &&
                     !(dx.vec && c.T <= 64);
  const bool rows = small && !curved && c.T <= 1024;  // db from dy's rows, without chunks
  if (curved || (c.db && !rows)) {
    const hipError_t e = act_grad_of<Tr>(c, c.db && !small, s);
    if (e != hipSuccess) return e;
  }
  if (small) {
    const int64_t n_w = w.G * cdiv(w.N, kSmall) * cdiv(w.K, kSmall), n_d = xcd_grid(cdiv(dx.P, kSmall) * cdiv(dx.K, kSmall)), n_c = c.db ? cdiv(c.N, 64) : 0;
    const dim3 grid((unsigned)(n_w + n_d + n_c));
    if (dx.vec) linear_grad_small_kernel<Tr, true, Args><<<grid, 256, 0, s>>>(dx, w, c, rows, (int)n_w, (int)n_d);
    else linear_grad_small_kernel<Tr, false, Args><<<grid, 256, 0, s>>>(dx, w, c, rows, (int)n_w, (int)n_d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else {
    if (dx.out && c.T > 0) {
      const hipError_t e = launch_vec<Tr, kDgrad, Args>(dx, s);
      if (e != hipSuccess) return e;
    }
    if (dw.out) {
      const hipError_t e = launch_vec<Tr, kWgrad, Args>(w, s);
      if (e != hipSuccess) return e;
    }
  }
  if (cut) {
    const int64_t n = (int64_t)dw.N * dw.K;
    add_parts_kernel<Tr><<<dim3((unsigned)cdiv(n, 1024)), 256, 0, s>>>(parts, dw.G, n, dw.out, dw.out_f32, dw.accumulate);
  }
  return hipGetLastError();
}

}  // namespace

ColumnChunks column_chunks(int32_t T, int32_t cols) {
  // about 2048 workgroups of 256 columns, of eight rows at least
  const int64_t blocks = cdiv(cols, 256), most = blocks >= 2048 ? 1 : 2048 / blocks;
  int64_t rows = cdiv(T > 0 ? T : 1, most);
  rows = cdiv(rows, 8) * 8;
  return {(int32_t)rows, (int32_t)cdiv(T, rows)};
}

RowParts weight_parts(int32_t T, int32_t N, int32_t K, bool wide) {
  // The number of parts with the shortest time: that of the tiles, and of writing and reading the parts (4 TB/s) and another
  // launch; at most 128 MiB. 8192 rows, 512 x 512 100 us uncut, 1024 x 1024 102.
  RowParts best = {T > 0 ? T : 1, 1};
  int64_t least = INT64_MAX;
  for (int32_t count = 1; count <= 32; count *= 2) {
    const int32_t rows = (int32_t)(cdiv(cdiv(T > 0 ? T : 1, count), kBR) * kBR);
    if (count > 1 && ((int64_t)(count - 1) * rows >= T || (int64_t)count * N * K > (int64_t)32 << 20)) break;
    int64_t t = wgrad_time(count > 1 ? rows : T, N, K, count, false);
    if (wide) t = wgrad_time(count > 1 ? rows : T, N, K, count, true) < t ? wgrad_time(count > 1 ? rows : T, N, K, count, true) : t;
    if (count > 1) t += 350 + (int64_t)count * N * K * 8 / 40000;
    if (t < least) {
      least = t;
      best = {count > 1 ? rows : (T > 0 ? T : 1), count};
    }
  }
  return best;
}

template <bool Gated>
hipError_t launch_linear(const LinearArgs<Gated> &a, bool fp16, hipStream_t s) {
  return fp16 ? linear_of<Fp16, Gated>(a, s) : linear_of<Bf16, Gated>(a, s);
}
template hipError_t launch_linear<false>(const LinearArgs<false> &, bool, hipStream_t);
template hipError_t launch_linear<true>(const LinearArgs<true> &, bool, hipStream_t);

hipError_t launch_linear_grad(const ActGradArgs &c, const DenseArgs &dx, const DenseArgs &dw, float *parts, bool fp16, hipStream_t s) {
  if (!grad_fits(c, dx, dw)) return hipErrorInvalidConfiguration;
  return fp16 ? linear_grad_of<Fp16, DenseArgs>(c, dx, dw, parts, s) : linear_grad_of<Bf16, DenseArgs>(c, dx, dw, parts, s);
}

hipError_t launch_linear_grad_split(const ActGradArgs &c, const SplitArgs &dx, const SplitArgs &dw, const HalvesArgs &w, const HalvesArgs &x,
                                    float *parts, bool fp16, bool bf16_parts, hipStream_t s) {
  if (!grad_fits(c, dx, dw)) return hipErrorInvalidConfiguration;
  for (const HalvesArgs *h : {&w, &x}) {
    if (!h->from || h->rows == 0) continue;
    const int64_t n = cdiv((int64_t)h->rows * cdiv(h->cols, 8), 256);
    halves_kernel<<<dim3((unsigned)(n < 8192 ? n : 8192)), 256, 0, s>>>(*h);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (bf16_parts) return linear_grad_of<Fp16InBf16, SplitArgs>(c, dx, dw, parts, s);
  return fp16 ? linear_grad_of<Fp16, SplitArgs>(c, dx, dw, parts, s) : linear_grad_of<Bf16, SplitArgs>(c, dx, dw, parts, s);
}

}  // namespace moe
