// Low-rank adapters of many requests beside a shared projection, and their
// gradients, for gfx950.
//
//   h[t] = scale_a A_a x[t],  y[t] = base[t] + B_a h[t]          a = adapter of t
//   g[t] = scale_a B_a^T dy[t],  dx[t] = dx_base[t] + A_a^T g[t]
//   dA_a = sum_t g[t] x[t]^T,  dB_a = sum_t dy[t] h[t]^T
//
// Rows come sorted by adapter (rows[], offsets[]); a workgroup takes up to 16
// or 32 rows of one adapter and forms both products of them, so h and g never leave
// the chip (but for the copies that dA and dB sum over). x A^T and dy B have
// 16-bit operands on both sides and run on the 16-bit matrix instructions. Their
// results h and g are fp32 and enter the second product whole: in bf16 as sums of three exact
// 16-bit parts, for which the 16-bit matrix instruction is still five times faster than the fp32
// one; in fp16, whose exponents cannot hold such parts, on the fp32 instruction. (8192 rows of 16
// adapters, 2048 x 4096, bf16 and fp16: rank 32 69 and 77 us, rank 64 98 and 119, rank 128 172 and 223.)
//
// Bound by memory, and in decode by the launch. 8192 rows, 16 adapters of rank 32, 2048 x 4096, bf16: 41 us
// (168 MB, 4.1 TB/s) where base and y stay in the last-level cache, 57 us where they do not. One row: 7 us of kernel.
// Gradients of 4096 rows, four adapters of rank 16, 2048 x 2048: 19 us for the rows, 16 us for the adapters.

#include "grouped_device.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kWaves = 8;                // waves of a workgroup
constexpr int kAdThreads = 64 * kWaves;

typedef s8 __attribute__((aligned(2))) s8_any;
// Eight elements of which `left` exist (no more are read).
__device__ __forceinline__ s8 load8(const uint16_t *p, int left, bool vec) {
  s8 v = {0, 0, 0, 0, 0, 0, 0, 0};
  if (left >= 8) {
    if (vec) v = *reinterpret_cast<const s8 *>(p);
    else v = *reinterpret_cast<const s8_any *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) v[i] = (short)p[i];
  }
  return v;
}

// The rows of a workgroup: places [at, at + n) of the sorted order, adapter e
// (-1: rows without one), or n <= 0. Rows without an adapter, which are only copied, come first,
// so that no copy starts when the other workgroups end. (Giving every XCD consecutive
// blocks, so that an adapter is read into one L2, measured slower: 70 against 62 us
// at 8192 rows; its workgroups then ask for the same lines at the same time.)
struct RowBlock { int e, at, n; };
template <int kAdRows>
__device__ __forceinline__ RowBlock find_rows(const int32_t *offsets, int adapters, int T, int m) {
  const int bare = min(max(offsets[adapters], 0), T);  // places from here on have no adapter
  const int copies = (T - bare + kAdRows - 1) / kAdRows;
  const GroupTile g = find_group(offsets, adapters, T, kAdRows, [&](int) { return m - copies; });
  RowBlock b;
  b.e = g.e;
  if (m < copies) {
    b.at = bare + m * kAdRows;
    b.n = min(kAdRows, T - b.at);
  } else {
    const int i0 = (m - copies - g.before) * kAdRows;
    b.at = g.first + i0;
    b.n = g.e < 0 ? 0 : min(kAdRows, g.count - i0);
  }
  return b;
}

// Row of x that place `i` of the block holds, or -1.
__device__ __forceinline__ int row_of(const int32_t *rows, const RowBlock &b, int i, int T) {
  if (i >= b.n) return -1;
  const int t = rows[b.at + i];
  return t >= 0 && t < T ? t : -1;
}

// LDS of a workgroup: the waves' partial first products ([wave][row block][rank tile][lane]),
// and before and after that each wave's own staging area.
template <int RT>
constexpr int kStageBytes = 16 * RT * 144;   // 16 RT rank rows of 64 columns, 16 bytes apart from each other's banks
template <int RT>
constexpr int kAdLds = kWaves * kStageBytes<RT>;

// Sum the waves' partial products and scale them. part[w][rb][rt][lane] holds
// row 16 rb + lane % 16, columns 16 rt + 4 (lane / 16) .. of wave w. The sums
// replace wave 0's partials. Columns from r on are zeros, also where the row's
// values are not finite (there 0 times them was added up).
template <int RB, int RT>
__device__ __forceinline__ void join_waves(f4 *part, const f4 (&acc)[RB][RT], float scale, int r) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < RT; ++j) part[((wave * RB + b) * RT + j) * 64 + lane] = acc[b][j];
  __syncthreads();
  for (int u = threadIdx.x; u < RB * RT * 64; u += kAdThreads) {
    f4 s = part[u];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += part[w * RB * RT * 64 + u];
    s *= scale;
    const int left = r - 16 * ((u >> 6) % RT) - 4 * ((u & 63) >> 4);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x >= left) s[x] = 0.f;
    part[u] = s;
  }
  __syncthreads();
}

// x A^T of the block's rows, inputs split over the waves: acc[b][j] holds row
// 16 b + p16, rank 16 j + 4 q4 .. of this wave's share.
template <typename Tr, int RB, int RT>
__device__ __forceinline__ void down_product(const uint16_t *x, int64_t ld_x, const int (&row)[RB], const uint16_t *A, int r,
                                             int K, bool vec, f4 (&acc)[RB][RT]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  constexpr int kDeep = RB * RT == 1 ? 8 : RT <= 2 ? 4 / RB : 1;  // steps whose loads are in flight together
  for (int k0 = 32 * wave; k0 < K; k0 += 32 * kWaves * kDeep) {
    s8 xv[kDeep][RB], av[kDeep][RT];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int k = k0 + 32 * kWaves * u + 8 * q4;
#pragma unroll
      for (int j = 0; j < RT; ++j) av[u][j] = load8(A + (int64_t)min(16 * j + p16, r - 1) * K + k, 16 * j + p16 < r ? K - k : 0, vec);
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {  // behind A's: the row numbers may still be on their way
      const int k = k0 + 32 * kWaves * u + 8 * q4;
#pragma unroll
      for (int b = 0; b < RB; ++b) xv[u][b] = load8(x + (int64_t)max(row[b], 0) * ld_x + k, row[b] >= 0 ? K - k : 0, vec);
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[b][j] = Tr::mfma(av[u][j], xv[u][b], acc[b][j]);
  }
}

// ------------------------------------------------------- the second product
// out[i][c] = sum_j h[i][j] m[j][c] with h fp32 in `part` as join_waves left it, and m 16-bit in operand
// registers: lane (p16, q4) holds column p16's eight ranks from 32 u + 8 q4 on in register set u, or, at
// one rank tile, from 8 (q4 & 1) on. times() gives the lane row p16 and columns 4 q4 .. of a 16 x 16 block.
__device__ __forceinline__ f4 mfma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

template <typename Tr, int RB, int RT> struct Middle;

// bf16: h is cut into three parts of eight bits each, exact: bf16 has fp32's exponents (only bits below 2^-133,
// those of values below 2^-110, are lost). The matrix instruction's 32 terms hold 32 ranks of a part,
// or, at one rank tile, 16 ranks of two parts, the last part in two halves.
template <int RB, int RT>
struct Middle<Bf16, RB, RT> {
  static constexpr int NM = RT / 2 ? RT / 2 : 1;
  static constexpr int kTerms = RT == 1 ? 2 : 3 * NM;  // instructions per block
  s8 v[RB][kTerms];  // operand of row p16

  static __device__ __forceinline__ float top8(float v) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u); }
  static __device__ __forceinline__ short bits(float v) { return (short)(__builtin_bit_cast(uint32_t, v) >> 16); }

  // The parts of v, leading bits first. Unless v is zero all of them have its sign and none is
  // zero, so that with an infinite weight each part's product is the infinity that v's is: where nothing is left for a part, it
  // takes half of the one before. Of an infinity or NaN every part is v.
  static __device__ __forceinline__ void cut(float v, float &a, float &b, float &c) {
    const bool finite = (__builtin_bit_cast(uint32_t, v) & 0x7f800000u) != 0x7f800000u;
    a = top8(v);
    float left = finite ? v - a : v;
    if (left == 0.f) a = left = 0.5f * a;
    b = top8(left);
    c = finite ? left - b : v;
    if (c == 0.f) b = c = 0.5f * b;
  }

  __device__ __forceinline__ void read(const f4 *part) {
    const int lane = threadIdx.x & 63, p16 = lane & 15, q4 = lane >> 4;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int u = 0; u < NM; ++u) {
        const int j = RT == 1 ? 8 * (q4 & 1) : 32 * u + 8 * q4;  // first of this lane's eight ranks
        const f4 *q = part + (r * RT + (j >> 4)) * 64 + p16 + 16 * ((j >> 2) & 3);
        const f4 lo = q[0], hi = q[16];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float a, b, c;
          cut(x < 4 ? lo[x & 3] : hi[x & 3], a, b, c);
          if constexpr (RT == 1) {
            v[r][0][x] = bits(q4 >> 1 ? b : a);
            v[r][1][x] = bits(0.5f * c);
          } else {
            v[r][u][x] = bits(a);
            v[r][NM + u][x] = bits(b);
            v[r][2 * NM + u][x] = bits(c);
          }
        }
      }
  }
  __device__ __forceinline__ f4 times(int b, const s8 (&m)[NM]) const {
    f4 acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kTerms; ++u) acc = Bf16::mfma(m[u % NM], v[b][u], acc);
    return acc;
  }
};

// fp16: the fp32 matrix instruction, on h as it is and the columns' values widened. fp16 parts would not
// do: fp16 spans 40 binary orders, so a rank whose h lies far below its row's largest would lose its bits,
// though its column may be the only one that another result takes. Instruction x takes rank 8 q4 + x of each 32, or,
// at one rank tile, rank 8 (q4 & 1) + 4 (q4 / 2) + x.
template <int RB, int RT>
struct Middle<Fp16, RB, RT> {
  static constexpr int NM = RT / 2 ? RT / 2 : 1, kEach = RT == 1 ? 4 : 8;
  float v[RB][NM * kEach];  // operand of row p16

  __device__ __forceinline__ void read(const f4 *part) {
    const int lane = threadIdx.x & 63, p16 = lane & 15, q4 = lane >> 4;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int u = 0; u < NM; ++u) {
        const int j = RT == 1 ? 8 * (q4 & 1) + 4 * (q4 >> 1) : 32 * u + 8 * q4;  // first of this lane's ranks
        const f4 *q = part + (b * RT + (j >> 4)) * 64 + p16 + 16 * ((j >> 2) & 3);
#pragma unroll
        for (int y = 0; y < kEach / 4; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) v[b][u * kEach + 4 * y + x] = q[16 * y][x];
      }
  }
  __device__ __forceinline__ f4 times(int b, const s8 (&m)[NM]) const {
    const bool upper = (threadIdx.x & 32) != 0;
    f4 acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NM; ++u) {
      u4 w = __builtin_bit_cast(u4, m[u]);
      if (RT == 1) {
        w[0] = upper ? w[2] : w[0];
        w[1] = upper ? w[3] : w[1];
      }
#pragma unroll
      for (int x = 0; x < kEach; ++x)
        acc = mfma32(Fp16::to((uint16_t)(w[x >> 1] >> (16 * (x & 1)))), v[b][u * kEach + x], acc);
    }
    return acc;
  }
};

// Eight consecutive values of base or y from element `at` on, of which `left` exist, as they lie in memory.
template <bool F32> struct Eight { u4 v[F32 ? 2 : 1]; };
template <bool F32>
__device__ __forceinline__ Eight<F32> load_out(const void *p, int64_t at, bool vec, int left) {
  Eight<F32> e;
  if constexpr (F32) {
    const uint32_t *q = static_cast<const uint32_t *>(p) + at;
    if (vec && left >= 8) {
      e.v[0] = reinterpret_cast<const u4 *>(q)[0];
      e.v[1] = reinterpret_cast<const u4 *>(q)[1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e.v[i >> 2][i & 3] = i < left ? q[i] : 0u;
    }
  } else {
    e.v[0] = __builtin_bit_cast(u4, load8(static_cast<const uint16_t *>(p) + at, left, vec));
  }
  return e;
}
template <typename Tr, bool F32>
__device__ __forceinline__ float value_of(const Eight<F32> &e, int i) {
  if constexpr (F32) return __builtin_bit_cast(float, (uint32_t)e.v[i >> 2][i & 3]);
  else return Tr::to((uint16_t)(e.v[0][i >> 1] >> (16 * (i & 1))));
}
template <typename Tr, bool F32>
__device__ __forceinline__ void store_out(void *p, int64_t at, bool vec, int left, const float *f) {
  if constexpr (F32) {
    float *q = static_cast<float *>(p) + at;
    if (vec && left >= 8) {
      reinterpret_cast<f4 *>(q)[0] = f4{f[0], f[1], f[2], f[3]};
      reinterpret_cast<f4 *>(q)[1] = f4{f[4], f[5], f[6], f[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = f[i];
    }
  } else {
    uint16_t *q = static_cast<uint16_t *>(p) + at;
    if (vec && left >= 8) {
      u4 v;
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = (uint32_t)Tr::from(f[2 * x]) | (uint32_t)Tr::from(f[2 * x + 1]) << 16;
      *reinterpret_cast<u4 *>(q) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = Tr::from(f[i]);
    }
  }
}

// What the second product adds to and writes.
struct OutRows {
  const void *base;
  int64_t ld_base;
  void *out;
  int64_t ld_out;
  bool vec;
};

// A wave's 64 columns from n0 on: four 16-column blocks. Block c, operand row m
// is column 32 (c / 2) + 8 (m / 4) + 4 (c % 2) + m % 4, so that a lane
// ends with two runs of eight columns, n0 + 8 q4 and n0 + 32 + 8 q4.
template <bool F32, int RB>
__device__ __forceinline__ void load_base(const OutRows &o, const int (&row)[RB], int n0, int end, Eight<F32> (&f)[RB][2]) {
  const int q4 = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = n0 + 32 * h + 8 * q4;
      f[b][h] = load_out<F32>(o.base, (int64_t)max(row[b], 0) * o.ld_base + col, o.vec, o.base && row[b] >= 0 ? end - col : 0);
    }
}
template <typename Tr, bool F32, int RB, int RT>
__device__ __forceinline__ void finish(const OutRows &o, const int (&row)[RB], int n0, int end, const Middle<Tr, RB, RT> &h,
                                       const s8 (&m)[4][RT / 2 ? RT / 2 : 1], const Eight<F32> (&base)[RB][2]) {
  const int q4 = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float f[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f4 acc = h.times(b, m[2 * x + c]);
#pragma unroll
        for (int y = 0; y < 4; ++y) f[4 * c + y] = value_of<Tr, F32>(base[b][x], 4 * c + y) + acc[y];
      }
      const int col = n0 + 32 * x + 8 * q4;
      if (row[b] >= 0 && col < end) store_out<Tr, F32>(o.out, (int64_t)row[b] * o.ld_out + col, o.vec, end - col, f);
    }
}

// Rows without an adapter: out = base. A wave copies every eighth row, 512 columns at a time.
template <typename Tr, bool F32, int RB>
__device__ __forceinline__ void copy_rows(const OutRows &o, const int (&row)[RB], int begin, int end) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  constexpr int kDeep = 4;
#pragma unroll
  for (int b = 0; b < RB; ++b)
    for (int i = wave; i < 16; i += kWaves) {
      const int r = __shfl(row[b], i);
      if (r < 0) continue;
      for (int n0 = begin + 8 * lane; n0 < end; n0 += 512 * kDeep) {
        Eight<F32> e[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
          e[u] = load_out<F32>(o.base, (int64_t)r * o.ld_base + n0 + 512 * u, o.vec, o.base ? end - n0 - 512 * u : 0);
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          float f[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) f[x] = value_of<Tr, F32>(e[u], x);
          if (n0 + 512 * u < end) store_out<Tr, F32>(o.out, (int64_t)r * o.ld_out + n0 + 512 * u, o.vec, end - n0 - 512 * u, f);
        }
      }
    }
}

// Forward. Every slice of y's columns forms h for itself.
template <typename Tr, int RT, int RB, bool F32>
__global__ __launch_bounds__(kAdThreads, RT <= 2 ? 4 : 2) void adapter_kernel(AdapterArgs a, int slice) {
  constexpr int NM = RT / 2 ? RT / 2 : 1;
  __shared__ __attribute__((aligned(16))) f4 s_part[kWaves * RB * RT * 64];
  const RowBlock blk = find_rows<16 * RB>(a.offsets, a.n, a.T, blockIdx.x);
  if (blk.n <= 0) return;
  const bool same = a.base == a.y && a.ld_base == a.ld_y;
  if (blk.e < 0 && same) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  int row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = row_of(a.rows, blk, 16 * b + p16, a.T);
  const OutRows o{a.base, a.ld_base, a.y, a.ld_y, a.vec_y != 0};
  const int begin = blockIdx.y * slice, end = min(a.N, begin + slice);
  if (blk.e < 0) {
    copy_rows<Tr, F32, RB>(o, row, begin, end);
    return;
  }
  const uint16_t *B = a.B + (int64_t)blk.e * a.N * a.r;
  s8 m[4][NM];
  Eight<F32> f[RB][2];
  auto ask = [&](int n0) {  // a chunk's B and base
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int n = n0 + 32 * (c >> 1) + 8 * (p16 >> 2) + 4 * (c & 1) + (p16 & 3);
#pragma unroll
      for (int u = 0; u < NM; ++u) {
        const int j = RT == 1 ? 8 * (q4 & 1) : 32 * u + 8 * q4;
        m[c][u] = load8(B + (int64_t)n * a.r + j, n < end ? a.r - j : 0, a.vec_b);
      }
    }
    load_base<F32, RB>(o, row, n0, end, f);
  };
  int n0 = begin + 64 * wave;
  if (n0 < end) ask(n0);  // the first chunk's, beside the first product
  f4 acc[RB][RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[b][j] = f4{0.f, 0.f, 0.f, 0.f};
  down_product<Tr, RB, RT>(a.x, a.ld_x, row, a.A + (int64_t)blk.e * a.r * a.K, a.r, a.K, a.vec_x, acc);
  join_waves<RB, RT>(s_part, acc, a.scale ? a.scale[blk.e] : 1.f, a.r);
  Middle<Tr, RB, RT> h;
  h.read(s_part);
  for (; n0 < end; n0 += 64 * kWaves) {
    finish<Tr, F32, RB, RT>(o, row, n0, end, h, m, f);
    if (n0 + 64 * kWaves < end) ask(n0 + 64 * kWaves);
  }
}

// Four consecutive values of column `c` of a tile of 16-bit rows of `bytes` bytes in LDS, for the lane's place in
// its 16: rows row0 + 0 .. 3 of column c0 + step (p16 / 4) + p16 % 4.
__device__ __forceinline__ s4 column4(const uint8_t *t, int bytes, int row0, int c0, int step) {
  const int p16 = threadIdx.x & 15;
  return read_lds_tr(t + (row0 + (p16 >> 2)) * bytes + 2 * (c0 + step * (p16 & 3)));
}

// Gradient by rows: g and h of every sorted place into the workspace, and dx.
// Both operands that lie across (B for g, A for dx) pass through a staging area of the wave.
template <typename Tr, int RT, int RB, bool F32>
__global__ __launch_bounds__(kAdThreads, RT <= 2 ? 4 : 2) void adapter_rows_grad_kernel(AdapterGradArgs a, int slice) {
  constexpr int NM = RT / 2 ? RT / 2 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t s_mem[kAdLds<RT>];
  static_assert(kAdLds<RT> >= kWaves * RB * RT * 1024, "the partial products fit");
  f4 *s_part = reinterpret_cast<f4 *>(s_mem);
  const RowBlock blk = find_rows<16 * RB>(a.offsets, a.n, a.T, blockIdx.x);
  if (blk.n <= 0) return;
  const bool same = a.dx_base == a.dx && a.ld_dx_base == a.ld_dx;
  if (blk.e < 0 && (!a.dx || same)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  int row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = row_of(a.rows, blk, 16 * b + p16, a.T);
  const OutRows o{a.dx_base, a.ld_dx_base, a.dx, a.ld_dx, a.vec_dx != 0};
  const int begin = blockIdx.y * slice, end = min(a.K, begin + slice);
  // with dB, the last blockIdx.y forms h, the others g and their slice of dx
  const bool for_h = a.dB && blockIdx.y + 1 == gridDim.y;
  if (blk.e < 0) {
    if (a.dx && !for_h) copy_rows<Tr, F32, RB>(o, row, begin, end);
    return;
  }
  uint8_t *mine = s_mem + wave * kStageBytes<RT>;
  const uint16_t *A = a.A + (int64_t)blk.e * a.r * a.K;
  const uint16_t *B = a.B + (int64_t)blk.e * a.N * a.r;
  const float scale = a.scale ? a.scale[blk.e] : 1.f;
  // the block's h or g into the workspace
  auto keep = [&](float *dst) {
    if (!dst) return;
    for (int u = threadIdx.x; u < RB * RT * 64; u += kAdThreads) {
      const int l = u & 63, j = (u >> 6) % RT, b = (u >> 6) / RT;
      const int i = 16 * b + (l & 15);
      if (i < blk.n) *reinterpret_cast<f4 *>(dst + ((int64_t)(blk.at + i) * RT + j) * 16 + 4 * (l >> 4)) = s_part[u];
    }
  };
  f4 acc[RB][RT];
  auto clear = [&]() {
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[b][j] = f4{0.f, 0.f, 0.f, 0.f};
  };
  if (for_h) {
    clear();
    down_product<Tr, RB, RT>(a.x, a.ld_x, row, A, a.r, a.K, a.vec_x, acc);
    join_waves<RB, RT>(s_part, acc, scale, a.r);
    keep(a.h);
    return;
  }
  // g: 32 columns of dy at a time, split over the waves; 32 rows of B are staged as 16 RT ranks each
  clear();
  constexpr int kDeep = RT <= 2 ? 4 / RB : 1;  // steps whose loads are in flight together
  static_assert(RT * 1024 <= kStageBytes<RT>, "a step of B fits");
  for (int n0 = 32 * wave; n0 < a.N; n0 += 32 * kWaves * kDeep) {
    s8 dv[kDeep][RB], bv[kDeep][RT];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int n1 = n0 + 32 * kWaves * u, n = n1 + 8 * q4;
#pragma unroll
      for (int b = 0; b < RB; ++b) dv[u][b] = load8(a.dy + (int64_t)max(row[b], 0) * a.ld_dy + n, row[b] >= 0 ? a.N - n : 0, a.vec_dy);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int unit = lane + 64 * i, nb = n1 + unit / (2 * RT), j = 8 * (unit % (2 * RT));
        bv[u][i] = load8(B + (int64_t)nb * a.r + j, nb < a.N ? a.r - j : 0, a.vec_b);
      }
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
#pragma unroll
      for (int i = 0; i < RT; ++i) *reinterpret_cast<s8 *>(mine + 16 * (lane + 64 * i)) = bv[u][i];
      wave_sync();
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const s4 lo = column4(mine, 32 * RT, 8 * q4, 16 * j, 4), hi = column4(mine, 32 * RT, 8 * q4 + 4, 16 * j, 4);
        const s8 w = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b][j] = Tr::mfma(w, dv[u][b], acc[b][j]);
      }
      wave_sync();
    }
  }
  join_waves<RB, RT>(s_part, acc, scale, a.r);
  if (blockIdx.y == 0) keep(a.g);  // dA's factor
  if (!a.dx) return;
  Middle<Tr, RB, RT> g;
  g.read(s_part);
  __syncthreads();  // the staging areas take the partials' place
  for (int k0 = begin + 64 * wave; k0 < end; k0 += 64 * kWaves) {
    Eight<F32> f[RB][2];
    s8 av[2 * RT];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) {
      const int unit = lane + 64 * i, j = unit >> 3, col = k0 + 8 * (unit & 7);
      av[i] = load8(A + (int64_t)j * a.K + col, j < a.r ? end - col : 0, a.vec_x);
    }
    load_base<F32, RB>(o, row, k0, end, f);
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) {
      const int unit = lane + 64 * i;
      *reinterpret_cast<s8 *>(mine + (unit >> 3) * 144 + 16 * (unit & 7)) = av[i];
    }
    wave_sync();
    s8 m[4][NM];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int u = 0; u < NM; ++u) {
        const int j = RT == 1 ? 8 * (q4 & 1) : 32 * u + 8 * q4, c0 = 32 * (c >> 1) + 4 * (c & 1);
        const s4 lo = column4(mine, 144, j, c0, 8), hi = column4(mine, 144, j + 4, c0, 8);
        m[c][u] = s8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
    wave_sync();
    finish<Tr, F32, RB, RT>(o, row, k0, end, g, m, f);
  }
}

// Gradient of the adapters: out[c][j] = sum over the adapter's rows of
// v[row][c] * m[place][j], v = x (dA, c = k) or dy (dB, c = n), m = g or h.
// Split: a workgroup owns 64 columns of one adapter; its waves take every eighth
// group of four rows, and join in LDS. Else every wave owns 64 columns and takes all rows,
// for adapters of few rows, where the join would be most of the work. Lane (p16, q4) reads four consecutive columns 4 p16 .. of
// row q4, and the fp32 matrix instruction number x takes column 4 p16 + x. Rows are asked for
// kRowsDeep groups at a time, their numbers one batch earlier.
constexpr int kRowsDeep = 8;
template <typename Tr, int RT, bool Split>
__global__ __launch_bounds__(kAdThreads) void adapter_weights_grad_kernel(AdapterGradArgs a, int tiles_a, int tiles_all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  const int e = blockIdx.x / tiles_all;
  int tile = blockIdx.x - e * tiles_all;
  const bool is_a = tile < tiles_a;
  if (!is_a) tile -= tiles_a;
  const uint16_t *v = is_a ? a.x : a.dy;
  const int64_t ld = is_a ? a.ld_x : a.ld_dy;
  const float *m = is_a ? a.g : a.h;
  const int C = is_a ? a.K : a.N;
  const bool vec = is_a ? a.vec_x : a.vec_dy;
  const int c0 = 64 * (Split ? tile : kWaves * tile + wave);
  if (c0 >= C) return;  // only without Split, which has no barrier
  constexpr int kApart = Split ? 4 * kWaves : 4;  // rows from one of a wave's groups to the next
  const int own = q4 + (Split ? 4 * wave : 0);
  const int first = min(max(a.offsets[e], 0), a.T);
  const int count = max(min(max(a.offsets[e + 1], 0), a.T) - first, 0);
  void *out = is_a ? a.dA : a.dB;
  if (count == 0 && a.accumulate) return;
  f4 acc[RT][4];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[j][x] = f4{0.f, 0.f, 0.f, 0.f};
  const int c = c0 + 4 * p16, left = C - c;
  int at[kRowsDeep];
  auto numbers = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kRowsDeep; ++u) {
      const int i = i0 + kApart * u + own;
      at[u] = i < count ? a.rows[first + i] : -1;
    }
  };
  numbers(0);
  for (int i0 = 0; i0 < count; i0 += kApart * kRowsDeep) {
    u2 vv[kRowsDeep];
    float mv[kRowsDeep][RT];
#pragma unroll
    for (int u = 0; u < kRowsDeep; ++u) {
      const int i = i0 + kApart * u + own;
      const bool ok = at[u] >= 0 && at[u] < a.T;
      const uint16_t *q = v + (int64_t)(ok ? at[u] : 0) * ld + c;
      vv[u] = u2{0u, 0u};
      if (ok && left >= 4 && vec) {
        vv[u] = *reinterpret_cast<const u2 *>(q);
      } else if (ok) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < left) vv[u][x >> 1] |= (uint32_t)q[x] << (16 * (x & 1));
      }
#pragma unroll
      for (int j = 0; j < RT; ++j) mv[u][j] = ok ? m[(int64_t)(first + i) * (16 * RT) + 16 * j + p16] : 0.f;
    }
    numbers(i0 + kApart * kRowsDeep);
#pragma unroll
    for (int u = 0; u < kRowsDeep; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float w = Tr::to((uint16_t)(vv[u][x >> 1] >> (16 * (x & 1))));
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[j][x] = mfma32(w, mv[u][j], acc[j][x]);
      }
  }
  // Block x of a rank tile has, in lane (p16, q4), rank p16 of columns
  // 4 (4 q4 + reg) + x: the four x are consecutive columns.
  auto put = [&](int i, int col, f4 sum) {
    if (i >= a.r || col >= C) return;
    const int64_t to = is_a ? ((int64_t)e * a.r + i) * a.K + col : ((int64_t)e * a.N + col) * a.r + i;
    if (is_a && a.vec_da) {
      if (a.g_f32) {
        f4 *w = reinterpret_cast<f4 *>(static_cast<float *>(out) + to);
        *w = a.accumulate ? sum + *w : sum;
      } else {
        *reinterpret_cast<u2 *>(static_cast<uint16_t *>(out) + to) = u2{(uint32_t)Tr::from(sum[0]) | (uint32_t)Tr::from(sum[1]) << 16,
                                                                        (uint32_t)Tr::from(sum[2]) | (uint32_t)Tr::from(sum[3]) << 16};
      }
      return;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (col + x >= C) break;
      const int64_t at1 = to + (is_a ? x : (int64_t)x * a.r);
      if (a.g_f32) {
        float *w = static_cast<float *>(out) + at1;
        *w = sum[x] + (a.accumulate ? *w : 0.f);
      } else {
        static_cast<uint16_t *>(out)[at1] = Tr::from(sum[x]);
      }
    }
  };
  if constexpr (!Split) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int reg = 0; reg < 4; ++reg)
        put(16 * j + p16, c0 + 4 * (4 * q4 + reg), f4{acc[j][0][reg], acc[j][1][reg], acc[j][2][reg], acc[j][3][reg]});
  } else {
    // Join the waves through LDS, up to four rank tiles at a time; a thread adds up the waves' four
    // values x of one (p16, q4, reg).
    constexpr int JT = RT < 4 ? RT : 4;
    __shared__ __attribute__((aligned(16))) f4 s_part[kWaves * JT * 4 * 64];
#pragma unroll
    for (int j0 = 0; j0 < RT; j0 += JT) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) s_part[((wave * JT + j) * 4 + x) * 64 + lane] = acc[j0 + j][x];
      __syncthreads();
      for (int t = threadIdx.x; t < JT * 256; t += kAdThreads) {
        // neighbours: dA's columns, dB's ranks
        const int l = is_a ? (t >> 4 & 15) + 16 * (t >> 2 & 3) : (t & 15) + 16 * (t >> 6 & 3), reg = is_a ? t & 3 : t >> 4 & 3, j = t >> 8;
        f4 sum = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
          for (int x = 0; x < 4; ++x) sum[x] += reinterpret_cast<const float *>(&s_part[((w * JT + j) * 4 + x) * 64 + l])[reg];
        put(16 * (j0 + j) + (l & 15), c0 + 4 * (4 * (l >> 4) + reg), sum);
      }
    }
  }
}

// Stable counting sort of the rows by adapter, in one workgroup: counts in
// LDS, then the rows in order, 1024 at a time; a row's place is its adapter's
// running start, plus the rows of the same adapter in earlier waves of the
// batch, plus those in earlier lanes of its wave. Bound by the chain of batches, 2 to 3 us each, and of
// a wave's distinct adapters: 64 rows of one adapter 5.7 us, of 64 8.7; 8192 rows of 16 adapters 20 (in runs) and 28 us
// (mixed), of 512 24 and 76; 65536 of 16 128 and 197. A plan serves all projections of a batch.
constexpr int kPlanThreads = 1024, kPlanWaves = 16;
__global__ __launch_bounds__(kPlanThreads) void adapter_plan_kernel(const int32_t *ids, int T, int n, int32_t *rows, int32_t *offsets) {
  __shared__ int32_t s_start[MOE_MAX_ADAPTERS + 1];
  __shared__ uint16_t s_wave[kPlanWaves][MOE_MAX_ADAPTERS + 1];
  __shared__ int32_t s_sum[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i <= n; i += kPlanThreads) s_start[i] = 0;
  for (int i = tid; i < kPlanWaves * (MOE_MAX_ADAPTERS + 1); i += kPlanThreads) (&s_wave[0][0])[i] = 0;
  __syncthreads();
  auto id_of = [&](int t) {
    const int v = ids[t];
    return v >= 0 && v < n ? v : n;  // n: no adapter, sorted behind the others
  };
  for (int t = tid; t < T; t += kPlanThreads) atomicAdd(&s_start[id_of(t)], 1);
  __syncthreads();
  // exclusive prefix sum over n + 1 <= 1025 counts: one per thread and the last by itself
  const int mine = tid <= n ? s_start[tid] : 0;
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(sum, d);
    if (lane >= d) sum += v;
  }
  if (lane == 63) s_sum[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += s_sum[w];
  if (tid <= n) {
    s_start[tid] = sum - mine;
    offsets[tid] = sum - mine;
  }
  if (n == kPlanThreads && tid == kPlanThreads - 1) {
    s_start[n] = sum;
    offsets[n] = sum;
  }
  __syncthreads();
  for (int t0 = 0; t0 < T; t0 += kPlanThreads) {
    const int t = t0 + tid;
    const int id = t < T ? id_of(t) : -1;
    // rank among the wave's lanes of the same adapter; the last of them writes the wave's count
    int rank = 0;
    uint64_t todo = __ballot(id >= 0);
    while (todo) {
      const int who = __shfl(id, __builtin_ctzll(todo));
      const uint64_t same = __ballot(id == who);
      if (id == who) {
        rank = __popcll(same & ((1ull << lane) - 1));
        if (rank == 0) s_wave[wave][id] = (uint16_t)__popcll(same);
      }
      todo &= ~same;
    }
    __syncthreads();
    int at = -1;
    if (id >= 0) {
      at = s_start[id] + rank;
      for (int w = 0; w < wave; ++w) at += s_wave[w][id];
      rows[at] = t;
    }
    __syncthreads();
    // the batch's counts move into the starts and are cleared for the next batch
    for (int i = tid; i <= n; i += kPlanThreads) {
      int c = 0;
      for (int w = 0; w < kPlanWaves; ++w) {
        c += s_wave[w][i];
        s_wave[w][i] = 0;
      }
      s_start[i] += c;
    }
    __syncthreads();
  }
}

// Column slices per row block so that about one workgroup a CU is launched,
// no slice shorter than one pass of the waves: every slice forms the first product again. One, two
// and four workgroups a CU, us: forward of 2048 rows of 8 adapters (rank 16, 2048 x 2048) 11.3, 15.7 and -, of 4096
// of 16 15.4, 19.5 and -; 8192 rows of 16 (rank 32, 2048 x 4096) 58, 58 and 66; gradients of 4096 rows of 4 42.6,
// 44.6 and 52. Half a workgroup a CU: 13.2 for the 2048 rows.
int slices_for(int64_t blocks, int cols) {
  const int64_t most = cdiv(cols, 64 * kWaves);
  int64_t want = cdiv(256, blocks);
  if (want > most) want = most;
  return (int)(want < 1 ? 1 : want);
}

int64_t row_blocks(int T, int n, int rows) {
  const int64_t used = (n < T ? n : T) + 1;
  return (T + used * (rows - 1)) / rows;
}

// Rows a workgroup, 16 or 32. 16 give more workgroups; 32 read the adapters
// half as often, which tells sooner at higher rank, and hold in one block the rows of most adapters where those have
// 8 to 24 on average. At 2048 x 2048, 16 against 32 rows, forward / gradients, us. Rank 16: 2048 rows of 8
// adapters 11.5 / 23.8 against 19.4 / 26.2; 4096 of 256 23.4 / 56.4 against 20.3 / 52.5, of 1024 50.8 / 182 against
// 54.2 / 190; 8192 of 32 26.2 / 61.6 against 35.0 / 60.9, of 512 44.2 / 107 against 35.9 / 104; 16384 of 8
// 40.8 / 86.6 against 39.3 / 82.6. Rank 64: 2048 of 8 20.4 / 42.3 against 25.3 / 52.7; 4096 of 64 48.6 / 101
// against 44.8 / 96; 8192 of 8 43.2 / 99 against 36.1 / 93. Rank 64 in fp16, where the fp32 instruction takes
// longer than the adapters' reading: 4096 of 64 57 / 105 against 58 / 111; 8192 of 8 78 / 137 against 85 / 146; 8192
// of 16 at 2048 x 4096 119 against 138; 1000 of 64 35 against 28; 32768 of 8 214 / 455 against 215 / 449.
template <typename Tr, int RT>
bool few_rows(int T, int n) {
  return T < (RT <= 2 || std::is_same_v<Tr, Fp16> ? 16384 : 4096) && (T < 8 * (int64_t)n || T > 24 * (int64_t)n);
}

template <typename Tr, int RT, int RB, bool F32>
hipError_t run_forward(const AdapterArgs &a, hipStream_t s) {
  const int64_t blocks = row_blocks(a.T, a.n, 16 * RB);
  const int slice = (int)(cdiv(a.N, (int64_t)slices_for(blocks, a.N) * 64) * 64), slices = (int)cdiv(a.N, slice);
  if (!grid_fits(blocks, kAdThreads)) return hipErrorInvalidConfiguration;
  adapter_kernel<Tr, RT, RB, F32><<<dim3((unsigned)blocks, (unsigned)slices), kAdThreads, 0, s>>>(a, slice);
  return hipGetLastError();
}
template <typename Tr, int RT>
hipError_t run_forward(const AdapterArgs &a, hipStream_t s) {
  if constexpr (RT < 8) {  // at eight rank tiles 32 rows' operands spill
    if (!few_rows<Tr, RT>(a.T, a.n)) return a.y_f32 ? run_forward<Tr, RT, 2, true>(a, s) : run_forward<Tr, RT, 2, false>(a, s);
  }
  return a.y_f32 ? run_forward<Tr, RT, 1, true>(a, s) : run_forward<Tr, RT, 1, false>(a, s);
}

template <typename Tr, int RT, int RB, bool F32>
hipError_t run_rows_grad(const AdapterGradArgs &a, hipStream_t s) {
  const int64_t blocks = row_blocks(a.T, a.n, 16 * RB);
  if (blocks == 0) return hipSuccess;
  const int slice = (int)(cdiv(a.K, (int64_t)(a.dx ? slices_for(blocks, a.K) : 1) * 64) * 64), slices = (int)cdiv(a.K, slice);
  if (!grid_fits(blocks, kAdThreads)) return hipErrorInvalidConfiguration;
  adapter_rows_grad_kernel<Tr, RT, RB, F32><<<dim3((unsigned)blocks, (unsigned)slices + (a.dB != nullptr)), kAdThreads, 0, s>>>(a, slice);
  return hipGetLastError();
}
template <typename Tr, int RT>
hipError_t run_grad(const AdapterGradArgs &a, hipStream_t s) {
  // Waves share an adapter's rows where there are many a adapter. Whole gradients at rank 16 and
  // 2048 x 2048, shared against not, us: 4096 rows of 16 adapters 37 / 47, of 64 62 / 47, of 256 155 / 63;
  // 8192 rows of 32 64 / 63, of 128 105 / 71, of 1024 567 / 205; 16384 rows of 8 87 / 188.
  const bool split = a.T > (int64_t)128 * a.n;
  const int cols = split ? 64 : 64 * kWaves;
  const int ta = a.dA ? (int)cdiv(a.K, cols) : 0, tb = a.dB ? (int)cdiv(a.N, cols) : 0;
  if (!grid_fits((int64_t)a.n * (ta + tb), kAdThreads)) return hipErrorInvalidConfiguration;
  hipError_t err;
  constexpr int kMore = RT < 8 ? 2 : 1;
  if (few_rows<Tr, RT>(a.T, a.n)) err = a.dx_f32 ? run_rows_grad<Tr, RT, 1, true>(a, s) : run_rows_grad<Tr, RT, 1, false>(a, s);
  else err = a.dx_f32 ? run_rows_grad<Tr, RT, kMore, true>(a, s) : run_rows_grad<Tr, RT, kMore, false>(a, s);
  if (err != hipSuccess || ta + tb == 0) return err;
  const dim3 grid((unsigned)((int64_t)a.n * (ta + tb)));
  if (split) adapter_weights_grad_kernel<Tr, RT, true><<<grid, kAdThreads, 0, s>>>(a, ta, ta + tb);
  else adapter_weights_grad_kernel<Tr, RT, false><<<grid, kAdThreads, 0, s>>>(a, ta, ta + tb);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_plan(const int32_t *row_adapter, int32_t T, int32_t n, int32_t *rows, int32_t *offsets, hipStream_t s) {
  adapter_plan_kernel<<<1, kPlanThreads, 0, s>>>(row_adapter, T, n, rows, offsets);
  return hipGetLastError();
}

hipError_t launch_adapter(const AdapterArgs &a, bool fp16, hipStream_t s) {
  switch (rank_tiles(a.r)) {
    case 1: return fp16 ? run_forward<Fp16, 1>(a, s) : run_forward<Bf16, 1>(a, s);
    case 2: return fp16 ? run_forward<Fp16, 2>(a, s) : run_forward<Bf16, 2>(a, s);
    case 4: return fp16 ? run_forward<Fp16, 4>(a, s) : run_forward<Bf16, 4>(a, s);
    default: return fp16 ? run_forward<Fp16, 8>(a, s) : run_forward<Bf16, 8>(a, s);
  }
}

hipError_t launch_adapter_grad(const AdapterGradArgs &a, bool fp16, hipStream_t s) {
  switch (rank_tiles(a.r)) {
    case 1: return fp16 ? run_grad<Fp16, 1>(a, s) : run_grad<Bf16, 1>(a, s);
    case 2: return fp16 ? run_grad<Fp16, 2>(a, s) : run_grad<Bf16, 2>(a, s);
    case 4: return fp16 ? run_grad<Fp16, 4>(a, s) : run_grad<Bf16, 4>(a, s);
    default: return fp16 ? run_grad<Fp16, 8>(a, s) : run_grad<Bf16, 8>(a, s);
  }
}

}  // namespace moe
