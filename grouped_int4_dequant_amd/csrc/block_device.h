// Device pieces shared by the operators of the block around the experts: runs
// of eight values of any type and alignment, sums over a wave, and the sigmoid.
#pragma once

#include "block_internal.h"
#include "grouped_device.h"

namespace moe {

// Global loads and stores of 16 bytes need the alignment of their elements only.
typedef u4 __attribute__((aligned(2))) u4_elem;
typedef f4 __attribute__((aligned(4))) f4_elem;

// Eight values as they lie in memory: 16-bit ones in lo, fp32 ones in lo and hi.
struct Raw8 {
  u4 lo, hi;
};

// Values at + 0 .. 7 of p, of which the first `left` exist (the others read as zeros).
// Whole: all eight, or (left <= 0) none.
template <bool F32, bool Whole = false>
__device__ __forceinline__ Raw8 load_raw8(const void *p, int64_t at, int left) {
  Raw8 v = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (Whole && left <= 0) return v;
  if constexpr (F32) {
    const float *q = static_cast<const float *>(p) + at;
    if (Whole || left >= 8) {
      v.lo = __builtin_bit_cast(u4, (f4) * reinterpret_cast<const f4_elem *>(q));
      v.hi = __builtin_bit_cast(u4, (f4) * reinterpret_cast<const f4_elem *>(q + 4));
    } else {
      uint32_t x[8];  // (all asked for before any is used)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = 0u;
        if (i < left) x[i] = __builtin_bit_cast(uint32_t, q[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v.lo[i] = x[i];
        v.hi[i] = x[4 + i];
      }
    }
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + at;
    if (Whole || left >= 8) {
      v.lo = *reinterpret_cast<const u4_elem *>(q);
    } else {
      uint32_t x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = 0u;
        if (i < left) x[i] = q[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v.lo[i] = x[2 * i] | x[2 * i + 1] << 16;
    }
  }
  return v;
}
template <typename Tr, bool F32>
__device__ __forceinline__ void widen8(const Raw8 &v, float *f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (F32) f[i] = __builtin_bit_cast(float, i < 4 ? v.lo[i] : v.hi[i - 4]);
    else f[i] = Tr::to((uint16_t)(v.lo[i >> 1] >> (16 * (i & 1))));
  }
}
// The same for an array whose type is known at run time.
template <typename Tr, bool Whole = false>
__device__ __forceinline__ void load8(const void *p, bool f32, int64_t at, int left, float *f) {
  if (f32) widen8<Tr, true>(load_raw8<true, Whole>(p, at, left), f);
  else widen8<Tr, false>(load_raw8<false, Whole>(p, at, left), f);
}

// Stores the first `left` of eight values, rounded to the array's type.
template <typename Tr, bool Whole = false>
__device__ __forceinline__ void store8(void *p, bool f32, int64_t at, int left, const float *f) {
  if (Whole && left <= 0) return;
  if (f32) {
    float *q = static_cast<float *>(p) + at;
    if (Whole || left >= 8) {
      *reinterpret_cast<f4_elem *>(q) = f4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f4_elem *>(q + 4) = f4{f[4], f[5], f[6], f[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = f[i];
    }
  } else {
    uint16_t *q = static_cast<uint16_t *>(p) + at;
    if (Whole || left >= 8) {
      u4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint32_t)Tr::from(f[2 * i]) | (uint32_t)Tr::from(f[2 * i + 1]) << 16;
      *reinterpret_cast<u4_elem *>(q) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = Tr::from(f[i]);
    }
  }
}

template <int Ctrl>
__device__ __forceinline__ float dpp_f32(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), Ctrl, 0xf, 0xf, false));
}
// Sum over the 64 lanes in a fixed order, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);   // lanes 1,0,3,2 of each four
  v += dpp_f32<0x4E>(v);   // 2,3,0,1
  v += dpp_f32<0x124>(v);  // four on, in each 16
  v += dpp_f32<0x128>(v);  // eight on: every lane holds its 16 lanes' sum
  auto lane = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l)); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// s(v) = 1 / (1 + e^-v) and 1 - s(v). e^-|v| is 2^(-|v| log2 e) with the constant (within 0.22 2^-24 of log2 e) and the product
// rounded, which is off by 1.25 |v| 2^-24 of itself at most, and the exponential's own 2^-23: for the small one of the two that
// is its relative error (with three 2^-24 more for the sum and the reciprocal), and nothing to the other.
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float v) {
  const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(v) * -1.44269504f);
  const float big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
  return v < 0.f ? Sigmoid{small, big} : Sigmoid{big, small};
}
// v s(v), by the same way without the case distinction: e^-v may be infinite, its reciprocal is then zero.
__device__ __forceinline__ float times_sigmoid(float v, float of) {
  return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(of * -1.44269504f));
}

}  // namespace moe
