// Low-rank adapters of many requests beside a shared projection, and their
// gradients, for gfx950.
//
//   h[t] = scale_a A_a x[t],  y[t] = base[t] + B_a h[t]          a = adapter of t
//   g[t] = scale_a B_a^T dy[t],  dx[t] = dx_base[t] + A_a^T g[t]
//   dA_a = sum_t g[t] x[t]^T,  dB_a = sum_t dy[t] h[t]^T
//
// Rows come sorted by adapter (rows[], offsets[]). x A^T and dy B have 16-bit operands on
// both sides and run on the 16-bit matrix instructions; their results h and g stay fp32, and the
// products they enter run on the fp32 matrix instruction, so that nothing is
// rounded between the two factors of an adapter.

#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kWaves = 8;                // waves of a workgroup
constexpr int kAdThreads = 64 * kWaves;
constexpr int kRowBlocks = 2;            // 16-row blocks of a workgroup
constexpr int kAdRows = 16 * kRowBlocks;

// Eight elements of which `left` exist (no more than eight are read).
__device__ __forceinline__ s8 load8(const uint16_t *p, int left, bool vec) {
  s8 v = {0, 0, 0, 0, 0, 0, 0, 0};
  if (vec) {
    if (left > 0) v = *reinterpret_cast<const s8 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) v[i] = (short)p[i];
  }
  return v;
}

// The rows of a workgroup: places [at, at + n) of the sorted order, adapter e
// (-1: rows without one), or n == 0.
struct RowBlock { int e, at, n; };
__device__ __forceinline__ RowBlock find_rows(const int32_t *offsets, int adapters, int T, int m) {
  const GroupTile g = find_group(offsets, adapters, T, kAdRows, [&](int) { return m; });
  RowBlock b;
  if (g.e >= 0) {
    b.e = g.e;
    const int i0 = (m - g.before) * kAdRows;
    b.at = g.first + i0;
    b.n = min(kAdRows, g.count - i0);
  } else {
    b.e = -1;
    const int64_t at = min(max(offsets[adapters], 0), T) + (int64_t)(m - g.total) * kAdRows;
    b.at = (int)min(at, (int64_t)T);
    b.n = min(kAdRows, T - b.at);
  }
  return b;
}

// Row of x that place `i` of the block holds, or -1.
__device__ __forceinline__ int row_of(const int32_t *rows, const RowBlock &b, int i, int T) {
  if (i >= b.n) return -1;
  const int t = rows[b.at + i];
  return t >= 0 && t < T ? t : -1;
}

// Sum the waves' partial products and scale them. part[w][rb][rt][lane] holds
// row 16 rb + lane % 16, columns 16 rt + 4 (lane / 16) .. of wave w. The sums
// replace wave 0's partials.
template <int RB, int RT>
__device__ __forceinline__ void join_waves(f4 *part, float scale) {
  __syncthreads();
  for (int u = threadIdx.x; u < RB * RT * 64; u += kAdThreads) {
    f4 s = part[u];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += part[w * RB * RT * 64 + u];
    part[u] = s * scale;
  }
  __syncthreads();
}

// x A^T of the block's rows, inputs split over the waves.
template <typename Tr, int RB, int RT>
__device__ __forceinline__ void down_product(const uint16_t *x, int64_t ld_x, const int (&row)[RB], const uint16_t *A, int r,
                                             int K, bool vec, f4 *part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  f4 acc[RB][RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[b][j] = f4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 32 * wave; k0 < K; k0 += 32 * kWaves) {
    const int k = k0 + 8 * q4;
    s8 xv[RB], av[RT];
#pragma unroll
    for (int b = 0; b < RB; ++b) xv[b] = load8(x + (int64_t)max(row[b], 0) * ld_x + k, row[b] >= 0 ? K - k : 0, vec);
#pragma unroll
    for (int j = 0; j < RT; ++j) av[j] = load8(A + (int64_t)min(16 * j + p16, r - 1) * K + k, 16 * j + p16 < r ? K - k : 0, vec);
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[b][j] = Tr::mfma(av[j], xv[b], acc[b][j]);
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < RT; ++j) part[((wave * RB + b) * RT + j) * 64 + lane] = acc[b][j];
}

__device__ __forceinline__ f4 mfma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// Sixteen consecutive values of base or y.
template <typename Tr>
__device__ __forceinline__ void load16(const void *p, int64_t at, bool f32, bool vec, int left, float *f) {
  if (f32) {
    const float *q = static_cast<const float *>(p) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (vec && left >= 16) {
        const f4 v = reinterpret_cast<const f4 *>(q)[i];
        f[4 * i] = v[0]; f[4 * i + 1] = v[1]; f[4 * i + 2] = v[2]; f[4 * i + 3] = v[3];
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) f[4 * i + x] = 4 * i + x < left ? q[4 * i + x] : 0.f;
      }
    }
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + at;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const s8 v = load8(q + 8 * i, left - 8 * i, vec && left >= 16);
#pragma unroll
      for (int x = 0; x < 8; ++x) f[8 * i + x] = Tr::to((uint16_t)v[x]);
    }
  }
}
template <typename Tr>
__device__ __forceinline__ void store16(void *p, int64_t at, bool f32, bool vec, int left, const float *f) {
  if (f32) {
    float *q = static_cast<float *>(p) + at;
    if (vec && left >= 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<f4 *>(q)[i] = f4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) q[i] = f[i];
    }
  } else {
    uint16_t *q = static_cast<uint16_t *>(p) + at;
    if (vec && left >= 16) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = (uint32_t)Tr::from(f[8 * i + 2 * x]) | (uint32_t)Tr::from(f[8 * i + 2 * x + 1]) << 16;
        reinterpret_cast<u4 *>(q)[i] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) q[i] = Tr::from(f[i]);
    }
  }
}

// Forward. blockIdx.x: block of rows, blockIdx.y: slice of 64 kWaves columns of y (every
// slice forms h for itself).
template <typename Tr, int RT>
__global__ __launch_bounds__(kAdThreads) void adapter_kernel(AdapterArgs a, int slice) {
  constexpr int RB = kRowBlocks;
  __shared__ __attribute__((aligned(16))) f4 s_part[kWaves * RB * RT * 64];
  const RowBlock blk = find_rows(a.offsets, a.n, a.T, blockIdx.x);
  if (blk.n <= 0) return;
  const bool same = a.base == a.y && a.ld_base == a.ld_y;
  if (blk.e < 0 && same) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  int row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = row_of(a.rows, blk, 16 * b + p16, a.T);
  f4 h[RB][RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < RT; ++j) h[b][j] = f4{0.f, 0.f, 0.f, 0.f};
  if (blk.e >= 0) {
    down_product<Tr, RB, RT>(a.x, a.ld_x, row, a.A + (int64_t)blk.e * a.r * a.K, a.r, a.K, a.vec_x, s_part);
    join_waves<RB, RT>(s_part, a.scale ? a.scale[blk.e] : 1.f);
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < RT; ++j) h[b][j] = s_part[(b * RT + j) * 64 + lane];
  }
  // wave's 64 columns: block c holds, as its row m, column 16 (m / 4) + 4 c +
  // m % 4, so that a lane ends with 16 consecutive columns of its row of y
  const uint16_t *B = a.B + (int64_t)max(blk.e, 0) * a.N * a.r;
  const int n_end = min(a.N, (int)(blockIdx.y + 1) * slice);
  for (int n0 = blockIdx.y * slice + 64 * wave; n0 < n_end; n0 += 64 * kWaves) {
    f4 acc[RB][4];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[b][c] = f4{0.f, 0.f, 0.f, 0.f};
    if (blk.e >= 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = n0 + 16 * (p16 >> 2) + 4 * c + (p16 & 3);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const int left = n < a.N ? a.r - (16 * j + 4 * q4) : 0;
          const uint16_t *q = B + (int64_t)n * a.r + 16 * j + 4 * q4;
          uint16_t w[4] = {0, 0, 0, 0};
          if (a.vec_b) {
            if (left > 0) {
              const u2 v = *reinterpret_cast<const u2 *>(q);
              w[0] = (uint16_t)v[0]; w[1] = (uint16_t)(v[0] >> 16); w[2] = (uint16_t)v[1]; w[3] = (uint16_t)(v[1] >> 16);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x < left) w[x] = q[x];
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b][c] = mfma32(Tr::to(w[x]), h[b][j][x], acc[b][c]);
        }
      }
    }
    const int col = n0 + 16 * q4;
    if (col >= n_end) continue;
    const int left = n_end - col;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (row[b] < 0) continue;
      float f[16];
      if (a.base) {
        load16<Tr>(a.base, (int64_t)row[b] * a.ld_base + col, a.y_f32, a.vec_y, left, f);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += acc[b][i >> 2][i & 3];
      store16<Tr>(a.y, (int64_t)row[b] * a.ld_y + col, a.y_f32, a.vec_y, left, f);
    }
  }
}

// Gradient by rows: g and h of every sorted place into the workspace, and dx.
template <typename Tr, int RT>
__global__ __launch_bounds__(kAdThreads) void adapter_rows_grad_kernel(AdapterGradArgs a, int slice) {
  constexpr int RB = kRowBlocks;
  __shared__ __attribute__((aligned(16))) f4 s_part[kWaves * RB * RT * 64];
  const RowBlock blk = find_rows(a.offsets, a.n, a.T, blockIdx.x);
  if (blk.n <= 0) return;
  const bool same = a.dx_base == a.dx && a.ld_dx_base == a.ld_dx;
  if (blk.e < 0 && (!a.dx || same)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p16 = lane & 15, q4 = lane >> 4;
  int row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = row_of(a.rows, blk, 16 * b + p16, a.T);
  f4 g[RB][RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < RT; ++j) g[b][j] = f4{0.f, 0.f, 0.f, 0.f};
  const uint16_t *A = a.A + (int64_t)max(blk.e, 0) * a.r * a.K;
  if (blk.e >= 0) {
    const float scale = a.scale ? a.scale[blk.e] : 1.f;
    // this workgroup's share of h and g in the workspace (slice 0 writes them)
    auto keep = [&](float *dst) {
      if (!dst || blockIdx.y) return;
      for (int u = threadIdx.x; u < RB * RT * 64; u += kAdThreads) {
        const int l = u & 63, j = (u >> 6) % RT, b = (u >> 6) / RT;
        const int i = 16 * b + (l & 15);
        if (i < blk.n) *reinterpret_cast<f4 *>(dst + ((int64_t)(blk.at + i) * RT + j) * 16 + 4 * (l >> 4)) = s_part[u];
      }
    };
    if (a.dB && blockIdx.y == 0) {
      down_product<Tr, RB, RT>(a.x, a.ld_x, row, A, a.r, a.K, a.vec_x, s_part);
      join_waves<RB, RT>(s_part, scale);
      keep(a.h);
      __syncthreads();
    }
    // g: dy rows by B, columns split over the waves; B lies across
    const uint16_t *B = a.B + (int64_t)blk.e * a.N * a.r;
    for (int n0 = 32 * wave; n0 < a.N; n0 += 32 * kWaves) {
      const int n = n0 + 8 * q4;
      s8 dv[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) dv[b] = load8(a.dy + (int64_t)max(row[b], 0) * a.ld_dy + n, row[b] >= 0 ? a.N - n : 0, a.vec_dy);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        s8 bv = {0, 0, 0, 0, 0, 0, 0, 0};
        if (16 * j + p16 < a.r) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (n + x < a.N) bv[x] = (short)B[(int64_t)(n + x) * a.r + 16 * j + p16];
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) g[b][j] = Tr::mfma(bv, dv[b], g[b][j]);
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < RT; ++j) s_part[((wave * RB + b) * RT + j) * 64 + lane] = g[b][j];
    join_waves<RB, RT>(s_part, scale);
    keep(a.g);
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < RT; ++j) g[b][j] = s_part[(b * RT + j) * 64 + lane];
  }
  if (!a.dx) return;
  // dx: a wave's 64 columns as in the forward kernel
  const int k_end = min(a.K, (int)(blockIdx.y + 1) * slice);
  for (int k0 = blockIdx.y * slice + 64 * wave; k0 < k_end; k0 += 64 * kWaves) {
    f4 acc[RB][4];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[b][c] = f4{0.f, 0.f, 0.f, 0.f};
    if (blk.e >= 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = k0 + 16 * (p16 >> 2) + 4 * c + (p16 & 3);
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i = 16 * j + 4 * q4 + x;
            const float w = i < a.r && k < a.K ? Tr::to(A[(int64_t)i * a.K + k]) : 0.f;
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b][c] = mfma32(w, g[b][j][x], acc[b][c]);
          }
      }
    }
    const int col = k0 + 16 * q4;
    if (col >= k_end) continue;
    const int left = k_end - col;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (row[b] < 0) continue;
      float f[16];
      if (a.dx_base) {
        load16<Tr>(a.dx_base, (int64_t)row[b] * a.ld_dx_base + col, a.dx_f32, a.vec_dx, left, f);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += acc[b][i >> 2][i & 3];
      store16<Tr>(a.dx, (int64_t)row[b] * a.ld_dx + col, a.dx_f32, a.vec_dx, left, f);
    }
  }
}

// Gradient of the adapters: out[c][j] = sum over the adapter's rows of
// v[row][c] * m[place][j], v = x (dA, c = k) or dy (dB, c = n), m = g or h.
// A workgroup owns 128 columns of one adapter and up to four 16-wide rank
// tiles; its waves take every eighth group of four rows. Lane (p16, q4) reads
// eight consecutive columns 8 p16 .. of row q4, and the matrix instruction
// number x takes column 8 p16 + x.
template <typename Tr, int RT>
__global__ __launch_bounds__(kAdThreads) void adapter_weights_grad_kernel(AdapterGradArgs a, int tiles_a, int tiles_all, int rank_tiles) {
  __shared__ __attribute__((aligned(16))) f4 s_part[kWaves / 2 * RT * 8 * 64];
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
  const int c0 = 128 * tile, j0 = 16 * RT * blockIdx.y, ldm = 16 * rank_tiles;
  const int first = min(max(a.offsets[e], 0), a.T);
  const int count = max(min(max(a.offsets[e + 1], 0), a.T) - first, 0);
  void *out = is_a ? a.dA : a.dB;
  if (count == 0 && a.accumulate) return;
  f4 acc[RT][8];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[j][x] = f4{0.f, 0.f, 0.f, 0.f};
  const int c = c0 + 8 * p16;
  for (int i = 4 * wave + q4; i < (count + 3) / 4 * 4; i += 4 * kWaves) {
    int t = -1;
    if (i < count) t = a.rows[first + i];
    const bool ok = t >= 0 && t < a.T;
    const s8 vv = load8(v + (int64_t)(ok ? t : 0) * ld + c, ok ? C - c : 0, vec);
    float mv[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) mv[j] = ok ? m[(int64_t)(first + i) * ldm + j0 + 16 * j + p16] : 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float f = Tr::to((uint16_t)vv[x]);
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j][x] = mfma32(f, mv[j], acc[j][x]);
    }
  }
  // join the waves: the upper half hands its sums to the lower half, three times
#pragma unroll
  for (int half = kWaves / 2; half; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int x = 0; x < 8; ++x) s_part[((wave - half) * RT * 8 + j * 8 + x) * 64 + lane] = acc[j][x];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[j][x] += s_part[(wave * RT * 8 + j * 8 + x) * 64 + lane];
    }
  }
  if (wave) return;
  // lane: rank column p16, columns c0 + 8 (4 q4 + reg) + x
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int i = j0 + 16 * j + p16;
    if (i >= a.r) continue;
#pragma unroll
    for (int reg = 0; reg < 4; ++reg)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int col = c0 + 8 * (4 * q4 + reg) + x;
        if (col >= C) continue;
        const int64_t at = is_a ? ((int64_t)e * a.r + i) * a.K + col : ((int64_t)e * a.N + col) * a.r + i;
        const float s = acc[j][x][reg];
        if (a.g_f32) {
          float *o = static_cast<float *>(out) + at;
          *o = s + (a.accumulate ? *o : 0.f);
        } else {
          static_cast<uint16_t *>(out)[at] = Tr::from(s);
        }
      }
  }
}

// Stable counting sort of the rows by adapter, in one workgroup: counts in
// LDS, then the rows in order, 1024 at a time; a row's place is its adapter's
// running start, plus the rows of the same adapter in earlier waves of the
// batch, plus those in earlier lanes of its wave.
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

// Column slices per row block so that about two workgroups a CU are launched,
// no slice shorter than one pass of the waves.
int slices_for(int64_t blocks, int cols) {
  const int64_t most = cdiv(cols, 64 * kWaves);
  int64_t want = cdiv(512, blocks);
  if (want > most) want = most;
  return (int)(want < 1 ? 1 : want);
}

int64_t row_blocks(int T, int n) {
  const int64_t used = (n < T ? n : T) + 1;
  return (T + used * (kAdRows - 1)) / kAdRows;
}

template <typename Tr, int RT>
hipError_t run_forward(const AdapterArgs &a, hipStream_t s) {
  const int64_t blocks = row_blocks(a.T, a.n);
  if (!grid_fits(blocks, kAdThreads)) return hipErrorInvalidConfiguration;
  const int slices = slices_for(blocks, a.N);
  const int slice = (int)(cdiv(a.N, (int64_t)slices * 64) * 64);
  adapter_kernel<Tr, RT><<<dim3((unsigned)blocks, (unsigned)cdiv(a.N, slice)), kAdThreads, 0, s>>>(a, slice);
  return hipGetLastError();
}

template <typename Tr, int RT>
hipError_t run_grad(const AdapterGradArgs &a, hipStream_t s) {
  const int64_t blocks = row_blocks(a.T, a.n);
  const int64_t weight_blocks = (int64_t)a.n * (cdiv(a.K, 128) + cdiv(a.N, 128));
  if (!grid_fits(blocks, kAdThreads) || !grid_fits(weight_blocks, kAdThreads)) return hipErrorInvalidConfiguration;
  if (blocks > 0) {
    const int slices = a.dx ? slices_for(blocks, a.K) : 1;
    const int slice = (int)(cdiv(a.K, (int64_t)slices * 64) * 64);
    adapter_rows_grad_kernel<Tr, RT><<<dim3((unsigned)blocks, (unsigned)cdiv(a.K, slice)), kAdThreads, 0, s>>>(a, slice);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (!a.dA && !a.dB) return hipSuccess;
  constexpr int WT = RT < 4 ? RT : 4;
  const int ta = a.dA ? (int)cdiv(a.K, 128) : 0, tb = a.dB ? (int)cdiv(a.N, 128) : 0;
  adapter_weights_grad_kernel<Tr, WT><<<dim3((unsigned)((int64_t)a.n * (ta + tb)), (unsigned)(RT / WT)), kAdThreads, 0, s>>>(a, ta, ta + tb, RT);
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
