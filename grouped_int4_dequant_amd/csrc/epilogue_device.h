// What follows the product of the matrix kernels: bias, activation and
// residual. Everything is formed in fp32 from the accumulated sum and rounded once.
#pragma once

#include "block_device.h"

#include <type_traits>

namespace moe {

constexpr float kGeluC = 7.978845608e-01f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// The curve that an activation puts a value (the gate's, if gated) through.
__device__ __forceinline__ float curve_of(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f || z != z ? z : 0.f;
    case MOE_ACT_SILU:
    case MOE_ACT_SWIGLU: return times_sigmoid(z, z);
    case MOE_ACT_GELU: return 0.5f * z * erfcf(z * -7.071067812e-01f);
    case MOE_ACT_GELU_TANH:
    case MOE_ACT_GEGLU: return times_sigmoid(z, 2.f * kGeluC * fmaf(kGeluA * z * z, z, z));  // (1 + tanh u) / 2 = s(2 u)
    default: return z;
  }
}
// The curve's derivative, and its value for the gated ones.
__device__ __forceinline__ float slope_of(int act, float z, float &value) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU:
    case MOE_ACT_SWIGLU: {
      const Sigmoid g = sigmoid_of(z);
      value = z * g.s;
      return g.s * fmaf(z, g.rest, 1.f);
    }
    case MOE_ACT_GELU: return 0.5f * erfcf(z * -7.071067812e-01f) + z * (3.989422804e-01f * __builtin_amdgcn_exp2f(z * z * -7.213475204e-01f));
    case MOE_ACT_GELU_TANH:
    case MOE_ACT_GEGLU: {
      const Sigmoid g = sigmoid_of(2.f * kGeluC * fmaf(kGeluA * z * z, z, z));
      value = z * g.s;
      const float both = g.s * g.rest;  // where it is zero the curve is straight, though z^2 may have overflowed
      return both == 0.f ? g.s : fmaf(z * both, 2.f * kGeluC * fmaf(3.f * kGeluA * z, z, 1.f), g.s);
    }
    default: return 1.f;
  }
}

typedef u2 __attribute__((aligned(2))) u2_elem;

// Up to four values at + 0 .. 3.
template <typename Tr>
__device__ __forceinline__ f4 load4(const void *p, bool f32, int64_t at, int left) {
  f4 v = {0.f, 0.f, 0.f, 0.f};
  if (f32) {
    const float *q = static_cast<const float *>(p) + at;
    if (left >= 4) return *reinterpret_cast<const f4_elem *>(q);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) v[i] = q[i];
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + at;
    if (left >= 4) {
      const u2 w = *reinterpret_cast<const u2_elem *>(q);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = Tr::to((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) v[i] = Tr::to(q[i]);
    }
  }
  return v;
}
template <typename Tr>
__device__ __forceinline__ void store4_of(void *p, bool f32, int64_t at, int left, f4 v) {
  if (f32) {
    float *q = static_cast<float *>(p) + at;
    if (left >= 4) {
      *reinterpret_cast<f4_elem *>(q) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) q[i] = v[i];
    }
  } else {
    uint16_t *q = static_cast<uint16_t *>(p) + at;
    if (left >= 4) {
      *reinterpret_cast<u2_elem *>(q) = u2{(uint32_t)Tr::from(v[0]) | (uint32_t)Tr::from(v[1]) << 16,
                                           (uint32_t)Tr::from(v[2]) | (uint32_t)Tr::from(v[3]) << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) q[i] = Tr::from(v[i]);
    }
  }
}

// What the epilogue reads for four results of a row, asked for ahead of their sums.
struct Extra4 {
  f4 bias, bias_u, res;
};
template <typename Tr, typename Args>
__device__ __forceinline__ Extra4 extra4(const Args &a, int row, int col, int left) {
  Extra4 e;
  if (a.bias) {
    e.bias = load4<Tr>(a.bias, a.bias_f32, col, left);
    if constexpr (Args::kGated) e.bias_u = load4<Tr>(a.bias, a.bias_f32, a.N / 2 + col, left);
  }
  if (a.res) e.res = load4<Tr>(a.res, a.out_f32, (int64_t)row * a.ld_res + col, left);
  return e;
}
// Four sums of result row `row`, from result column `col` on, of which `left` exist: z is the product
// (the gate's if gated), u the product that it multiplies.
template <typename Tr, typename Args>
__device__ __forceinline__ void finish4(const Args &a, int row, int col, int left, f4 z, f4 u, const Extra4 &e) {
  if (a.bias) {
    z += e.bias;
    if constexpr (Args::kGated) u += e.bias_u;
  }
  if (a.pre) {
    store4_of<Tr>(a.pre, false, (int64_t)row * a.ld_pre + col, left, z);
    if constexpr (Args::kGated) store4_of<Tr>(a.pre, false, (int64_t)row * a.ld_pre + a.N / 2 + col, left, u);
  }
  if (a.act != MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = curve_of(a.act, z[i]);
      if constexpr (Args::kGated) z[i] *= u[i];
    }
  }
  if (a.res) z += e.res;
  store4_of<Tr>(a.out, a.out_f32, (int64_t)row * a.ld_out + col, left, z);
}

// The same for eight.
template <typename Tr, typename Args>
__device__ __forceinline__ void finish8(const Args &a, int row, int col, int left, float (&z)[8], float (&u)[8], const float (&bias)[2][8], const Raw8 &res) {
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] += bias[0][i];
      if constexpr (Args::kGated) u[i] += bias[1][i];
    }
  }
  if (a.pre) {
    store8<Tr>(a.pre, false, (int64_t)row * a.ld_pre + col, left, z);
    if constexpr (Args::kGated) store8<Tr>(a.pre, false, (int64_t)row * a.ld_pre + a.N / 2 + col, left, u);
  }
  if (a.act != MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] = curve_of(a.act, z[i]);
      if constexpr (Args::kGated) z[i] *= u[i];
    }
  }
  if (a.res) {
    float f[8];
    if (a.out_f32) widen8<Tr, true>(res, f);
    else widen8<Tr, false>(res, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += f[i];
  }
  store8<Tr>(a.out, a.out_f32, (int64_t)row * a.ld_out + col, left, z);
}

// The results of a wide tile. A lane holds 16 consecutive columns of row p16 of each of its wave's 16-row blocks
// (gated: eight of the gate and the eight that it multiplies). The sums of a block pass through 4 KiB of LDS of the
// wave's own, so that eight lanes (gated: four) have a row's consecutive columns and arrays are read and
// stored as whole lines (gated: halves). The loop over blocks stays one: unrolled, the activations fill the instruction
// cache and the accumulators' last uses move to scratch.
template <typename Tr, int TI, typename Args>
__device__ __forceinline__ void finish_wide(const Args &a, int i0, int j0, int ni, int nj, f4 (&acc)[TI][4], uint8_t *mine) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave >> 2, wj = wave & 3, p16 = lane & 15, q4 = lane >> 4;
  constexpr int C = Args::kGated ? 32 : 64;  // result columns of a wave
  constexpr int X = C / 32;                  // rows of a block that a lane finishes
  const int g = Args::kGated ? lane & 3 : lane & 7, col = C * wj + 8 * g, left = nj - col;
  // unit u (four sums) of row r lies in slot u ^ r of sixteen
  auto unit = [&](int r, int u) __attribute__((always_inline)) { return reinterpret_cast<f4 *>(mine + 256 * r + 16 * (u ^ r)); };
  auto row_of = [&](int i, int x) __attribute__((always_inline)) { return 16 * (wi + 2 * i) + (Args::kGated ? lane >> 2 : 8 * x + (lane >> 3)); };
  float bias[2][8];
  if (a.bias) {
    load8<Tr>(a.bias, a.bias_f32, j0 + col, left, bias[0]);
    if constexpr (Args::kGated) load8<Tr>(a.bias, a.bias_f32, a.N / 2 + j0 + col, left, bias[1]);
  }
  Raw8 res[X];  // the residual, one block ahead
  auto ask = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int64_t at = (int64_t)(i0 + row_of(i, x)) * a.ld_res + j0 + col;
      const int n = row_of(i, x) < ni ? left : 0;
      if (a.out_f32) res[x] = load_raw8<true>(a.res, at, n);
      else res[x] = load_raw8<false>(a.res, at, n);
    }
  };
  if (a.res) ask(0);
#pragma unroll 1
  for (int i = 0; i < TI; ++i) {
    const int row0 = 16 * (wi + 2 * i);
    if (row0 >= ni) break;
#pragma unroll
    for (int s = 0; s < TI; ++s) {
      if (s != i) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) *unit(p16, Args::kGated ? 8 * (c >> 1) + 2 * q4 + (c & 1) : 4 * q4 + c) = acc[s][c];
    }
    wave_sync();
    Raw8 now[X];
#pragma unroll
    for (int x = 0; x < X; ++x) now[x] = res[x];
    if (a.res && i + 1 < TI) ask(i + 1);
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int r = row_of(i, x) - row0;
      float z[8], u[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f4 v = *unit(r, 2 * g + c);
#pragma unroll
        for (int y = 0; y < 4; ++y) z[4 * c + y] = v[y];
        if constexpr (Args::kGated) {
          const f4 w = *unit(r, 8 + 2 * g + c);
#pragma unroll
          for (int y = 0; y < 4; ++y) u[4 * c + y] = w[y];
        }
      }
      if (row0 + r < ni && left > 0) finish8<Tr>(a, i0 + row0 + r, j0 + col, left, z, u, bias, now[x]);
    }
    wave_sync();
  }
}

}  // namespace moe
