// The weighted combine of expert rows and its gradient, for gfx950.
//
//   y[t] = sum_j w[t][j] o[pos[t][j]] + add[t]
//   d_o[pos[t][j]] = w[t][j] dy[t],   dw[t][j] = <dy[t], o[pos[t][j]]>
//
// Both are bound by memory: every element is read once and used for one or two
// operations. Sums are held in fp32, slots in ascending order and `add` last.
// bf16, width 2048: 8192 tokens x 8 slots in 69 us, 4.4 TB/s; the gradient of 2048 tokens in
// 29.5 us, 4.8 TB/s (a copy of 1 GiB runs at 5.2 TB/s).

#include "grouped_device.h"

namespace moe {
namespace {

template <typename Tr>
__device__ __forceinline__ void unpack8(u4 v, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = Tr::to((uint16_t)v[i]);
    f[2 * i + 1] = Tr::to((uint16_t)(v[i] >> 16));
  }
}
template <typename Tr>
__device__ __forceinline__ u4 pack8(const float *f) {
  u4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (uint32_t)Tr::from(f[2 * i]) | (uint32_t)Tr::from(f[2 * i + 1]) << 16;
  return v;
}

// One thread owns eight columns of one token (one column without Vec).
template <typename Tr, bool Vec>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineRowsArgs a) {
  constexpr int C = Vec ? 8 : 1;
  const int units = (a.d + C - 1) / C;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = id / units;
  if (t >= a.T) return;
  const int c = (int)(id - t * units) * C;
  float sum[C];
#pragma unroll
  for (int i = 0; i < C; ++i) sum[i] = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int p = a.pos[t * a.k + j];
    if (p < 0 || p >= a.P) continue;
    const float w = a.w ? a.w[t * a.k + j] : 1.f;
    const uint16_t *o = a.o + (int64_t)p * a.ld_o + c;
    float f[C];
    if constexpr (Vec) unpack8<Tr>(*reinterpret_cast<const u4 *>(o), f); else f[0] = Tr::to(*o);
#pragma unroll
    for (int i = 0; i < C; ++i) sum[i] += w * f[i];
  }
  if (a.add) {
    float f[C];
    if (a.add_f32) {
      const float *q = static_cast<const float *>(a.add) + t * a.ld_add + c;
#pragma unroll
      for (int i = 0; i < C; ++i) f[i] = q[i];
    } else {
      const uint16_t *q = static_cast<const uint16_t *>(a.add) + t * a.ld_add + c;
      if constexpr (Vec) unpack8<Tr>(*reinterpret_cast<const u4 *>(q), f); else f[0] = Tr::to(*q);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) sum[i] += f[i];
  }
  if (a.y_f32) {
    float *q = static_cast<float *>(a.y) + t * a.ld_y + c;
    if constexpr (Vec) {
      *reinterpret_cast<f4 *>(q) = f4{sum[0], sum[1], sum[2], sum[3]};
      *reinterpret_cast<f4 *>(q + 4) = f4{sum[4], sum[5], sum[6], sum[7]};
    } else {
      q[0] = sum[0];
    }
  } else {
    uint16_t *q = static_cast<uint16_t *>(a.y) + t * a.ld_y + c;
    if constexpr (Vec) *reinterpret_cast<u4 *>(q) = pack8<Tr>(sum); else *q = Tr::from(sum[0]);
  }
}

// One wave per (token, slot) pair.
template <typename Tr, bool Vec>
__global__ __launch_bounds__(256) void combine_rows_grad_kernel(CombineRowsGradArgs a) {
  constexpr int C = Vec ? 8 : 1;
  const int lane = threadIdx.x & 63;
  const int64_t pair = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (pair >= (int64_t)a.T * a.k) return;
  const int64_t t = pair / a.k;
  const int p = a.pos[pair];
  const bool ok = p >= 0 && p < a.P;
  const float w = a.w ? a.w[pair] : 1.f;
  float dot = 0.f;
  if (ok) {
    for (int c = lane * C; c < a.d; c += 64 * C) {
      float g[C], f[C];
      const uint16_t *q = a.dy + t * a.ld_dy + c;
      if constexpr (Vec) unpack8<Tr>(*reinterpret_cast<const u4 *>(q), g); else g[0] = Tr::to(*q);
      if (a.dw) {
        const uint16_t *o = a.o + (int64_t)p * a.ld_o + c;
        if constexpr (Vec) unpack8<Tr>(*reinterpret_cast<const u4 *>(o), f); else f[0] = Tr::to(*o);
#pragma unroll
        for (int i = 0; i < C; ++i) dot += g[i] * f[i];
      }
      if (a.d_o) {
#pragma unroll
        for (int i = 0; i < C; ++i) g[i] *= w;
        uint16_t *o = a.d_o + (int64_t)p * a.ld_do + c;
        if constexpr (Vec) *reinterpret_cast<u4 *>(o) = pack8<Tr>(g); else *o = Tr::from(g[0]);
      }
    }
  }
  if (a.dw) {
#pragma unroll
    for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) a.dw[pair] = dot;
  }
}

}  // namespace

hipError_t launch_combine_rows(const CombineRowsArgs &a, bool fp16, hipStream_t s) {
  const int64_t n = (int64_t)a.T * cdiv(a.d, a.vec ? 8 : 1);
  if (!grid_fits(cdiv(n, 256), 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)cdiv(n, 256));
  if (fp16) {
    if (a.vec) combine_rows_kernel<Fp16, true><<<grid, 256, 0, s>>>(a); else combine_rows_kernel<Fp16, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.vec) combine_rows_kernel<Bf16, true><<<grid, 256, 0, s>>>(a); else combine_rows_kernel<Bf16, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_combine_rows_grad(const CombineRowsGradArgs &a, bool fp16, hipStream_t s) {
  if (!grid_fits(cdiv((int64_t)a.T * a.k, 4), 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)cdiv((int64_t)a.T * a.k, 4));
  if (fp16) {
    if (a.vec) combine_rows_grad_kernel<Fp16, true><<<grid, 256, 0, s>>>(a); else combine_rows_grad_kernel<Fp16, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.vec) combine_rows_grad_kernel<Bf16, true><<<grid, 256, 0, s>>>(a); else combine_rows_grad_kernel<Bf16, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
