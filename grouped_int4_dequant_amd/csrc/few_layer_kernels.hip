// A mixture-of-experts layer with 16-bit weights for a few tokens, for gfx950:
// two kernels.
//
//   ids, g = top-k of the logits     h[t][j] = silu(W_g x[t]) * (W_u x[t]) of expert ids[t][j]
//   y[t] = sum_j g[t][j] W_dn h[t][j] + shared + add[t]
//
// A decode batch has little use of each weight, so the bytes of the picked experts set the time.
//   gate/up  every workgroup repeats the top-k (a token a wave) and sorts the pairs (token,
//            slot) by expert in LDS; the first one leaves that for the second kernel. Then it walks
//            over items of 8 columns of h of one expert (or the shared one): 16 rows of W_gu,
//            eight of the gate and the eight that it multiplies, whose sums its eight waves share and join
//            in LDS, in order.
//   down     a workgroup owns 16 columns of y. Its waves take one expert after the other; what an
//            expert gives each of its pairs goes to LDS, and is added up there by token in slot order.
// Weights go straight from memory to operand registers and are read once; a matrix instruction
// takes 16 rows of W and up to 16 pairs (an expert with more reads its weights again from L2).

#include "block_device.h"
#include "topk_device.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kWaves = 8;

// Runs of eight 16-bit values; without Vec rows may end inside one.
template <bool Vec>
__device__ __forceinline__ s8 load_w(const uint16_t *p, int left) {
  if constexpr (Vec) {
    const s8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
    return left > 0 ? __builtin_bit_cast(s8, (u4) * reinterpret_cast<const u4_elem *>(p)) : zero;
  } else {
    return __builtin_bit_cast(s8, load_raw8<false>(p, 0, left).lo);
  }
}

struct FewLds {
  int32_t count[MOE_MAX_EXPERTS];    // pairs of each expert, then its place among the picked ones
  int32_t ids[kFewPairs];
  float gate[kFewPairs];
  int32_t expert[kFewPairs], start[kFewPairs + 1], pair[kFewPairs];
  int32_t fill[kFewPairs];
  int32_t used;
};

// Top-k of all tokens and the pairs sorted by expert, by one workgroup.
template <int VPL>
__device__ __forceinline__ void make_plan(const FewArgs &a, FewLds &s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pairs = a.T * a.k;
  for (int e = tid; e < a.E; e += 64 * kWaves) s.count[e] = 0;
  for (int t = wave; t < a.T; t += kWaves) {
    int id;
    float g;
    topk_wave<VPL>(a.logits + (int64_t)t * a.E, a.E, a.k, lane, id, g);
    if (lane < a.k) {
      s.ids[t * a.k + lane] = id;
      s.gate[t * a.k + lane] = g;
    }
  }
  __syncthreads();
  // (kFewPairs is the number of threads)
  const int mine = tid < pairs ? s.ids[tid] : -1;
  if (mine >= 0) atomicAdd(&s.count[mine], 1);
  __syncthreads();
  if (wave == 0) {
    // lane l has the experts of its run: their number and pairs, then what lies before it
    const int run = (a.E + 63) >> 6, e0 = min(lane * run, a.E), e1 = min(e0 + run, a.E);
    int n = 0, p = 0;
    for (int e = e0; e < e1; ++e) {
      n += s.count[e] > 0;
      p += s.count[e];
    }
    int ns = n, ps = p;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(ns, d), y = __shfl_up(ps, d);
      if (lane >= d) {
        ns += x;
        ps += y;
      }
    }
    if (lane == 63) {
      s.used = ns;
      s.start[ns] = ps;
    }
    int u = ns - n, at = ps - p;
    for (int e = e0; e < e1; ++e) {
      const int c = s.count[e];
      if (c == 0) continue;
      s.expert[u] = e;
      s.start[u] = at;
      s.fill[u] = at;
      s.count[e] = u++;
      at += c;
    }
  }
  __syncthreads();
  // the order of an expert's pairs is of no consequence: each is a column of its own in the matrix instructions
  if (mine >= 0) s.pair[atomicAdd(&s.fill[s.count[mine]], 1)] = tid;
  __syncthreads();
  if (blockIdx.x != 0) return;
  if (tid < pairs) {
    a.plan->pair[tid] = s.pair[tid];
    a.plan->gate[tid] = s.gate[tid];
    if (a.topk_ids) a.topk_ids[tid] = mine;
    if (a.topk_w) a.topk_w[tid] = s.gate[tid];
  }
  if (tid < s.used) a.plan->expert[tid] = s.expert[tid];
  if (tid <= s.used) a.plan->start[tid] = s.start[tid];
  if (tid == 0) {
    a.plan->used = s.used;
    a.plan->start[s.used] = s.start[s.used];
  }
}

// Inner values. bf16: three parts that add up to the fp32 value, each an array of `rows` rows;
// fp16: fp32 (its parts would leave fp16's range).
template <typename Tr>
__device__ __forceinline__ void store_inner(void *h, int64_t part, int64_t at, f4 v, int left) {
  if constexpr (std::is_same_v<Tr, Fp16>) {
    float *q = static_cast<float *>(h) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) q[i] = v[i];
  } else {
    uint16_t *q = static_cast<uint16_t *>(h) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= left) break;
      float rest = v[i];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        // cut off, not rounded: the rest keeps its sign and stays finite; infinities and NaN have none
        uint32_t b = __builtin_bit_cast(uint32_t, rest);
        const bool whole = (b & 0x7f800000u) != 0x7f800000u;
        if (!whole && (b & 0x007fffffu)) b |= 0x00400000u;  // NaN stays NaN
        q[p * part + i] = (uint16_t)(b >> 16);
        rest = whole ? rest - __builtin_bit_cast(float, b & 0xffff0000u) : 0.f;
      }
    }
  }
}

__device__ __forceinline__ float silu_of(float z) { return z * sigmoid_of(z).s; }

template <typename Tr, int VPL, bool Vec>
__global__ __launch_bounds__(64 * kWaves) void few_gate_up_kernel(FewArgs a) {
  __shared__ FewLds s;
  __shared__ __attribute__((aligned(16))) f4 s_part[2][kWaves][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;
  make_plan<VPL>(a, s);
  const int per = (a.f + 7) / 8, per_sh = (a.f_sh + 7) / 8;
  const int items = s.used * per + per_sh;
  int buf = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    // the shared expert's items come first
    const bool shared = item < per_sh;
    const int u = shared ? 0 : (item - per_sh) / per;
    const int c0 = 8 * (shared ? item : item - per_sh - u * per), f = shared ? a.f_sh : a.f;
    const uint16_t *W = shared ? a.sh_gu : a.gu + (int64_t)s.expert[u] * 2 * a.f * a.d;
    const int col = c0 + (p16 & 7);
    const uint16_t *w = W + (int64_t)(min(col, f - 1) + (p16 & 8 ? f : 0)) * a.d;  // columns past the last repeat it
    const int first = shared ? 0 : s.start[u], rows = shared ? a.T : s.start[u + 1] - first;
    for (int r0 = 0; r0 < rows; r0 += 16) {
      const bool ok = r0 + p16 < rows;
      const int pair = !ok ? 0 : shared ? r0 + p16 : s.pair[first + r0 + p16];
      const uint16_t *x = a.x + (int64_t)(shared ? pair : pair / a.k) * a.ld_x;
      f4 acc = {0.f, 0.f, 0.f, 0.f};
      constexpr int kDeep = 8;
      for (int k0 = 32 * wave; k0 < a.d; k0 += 32 * kWaves * kDeep) {
        s8 wv[kDeep], xv[kDeep];
#pragma unroll
        for (int y = 0; y < kDeep; ++y) {
          const int k = k0 + 32 * kWaves * y + 8 * q4;
          wv[y] = load_w<Vec>(w + k, a.d - k);
        }
#pragma unroll
        for (int y = 0; y < kDeep; ++y) {
          const int k = k0 + 32 * kWaves * y + 8 * q4;
          xv[y] = load_w<Vec>(x + k, ok ? a.d - k : 0);
        }
#pragma unroll
        for (int y = 0; y < kDeep; ++y) acc = Tr::mfma(wv[y], xv[y], acc);
      }
      s_part[buf][wave][lane] = acc;
      __syncthreads();
      if (wave == (item & (kWaves - 1))) {
        f4 v = s_part[buf][0][lane];
#pragma unroll
        for (int y = 1; y < kWaves; ++y) v += s_part[buf][y][lane];
        // lane: pair p16; rows 4 q4 .. of the 16: columns 4 q4 .. of the gate, and behind them what it multiplies
        f4 h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = silu_of(v[i]) * __shfl(v[i], (lane + 32) & 63);
        const int c = c0 + 4 * q4;
        if (ok && q4 < 2 && c < f) {
          if (shared) store_inner<Tr>(a.h_sh, (int64_t)a.T * a.pitch_sh, (int64_t)pair * a.pitch_sh + c, h, f - c);
          else store_inner<Tr>(a.h, (int64_t)a.T * a.k * a.pitch, (int64_t)pair * a.pitch + c, h, f - c);
        }
      }
      buf ^= 1;  // a wave may fill the next one while its last reader is at work; the barrier behind that ends both
    }
  }
}

// h of one pair, eight values from k on, times a run of W.
template <typename Tr, bool Vec>
struct Inner;
template <bool Vec>
struct Inner<Bf16, Vec> {
  s8 v[3];
  __device__ __forceinline__ void load(const void *h, int64_t part, int64_t at, int left) {
#pragma unroll
    for (int p = 0; p < 3; ++p) v[p] = load_w<Vec>(static_cast<const uint16_t *>(h) + p * part + at, left);
  }
  __device__ __forceinline__ f4 times(s8 w, f4 acc) const {
#pragma unroll
    for (int p = 0; p < 3; ++p) acc = Bf16::mfma(w, v[p], acc);
    return acc;
  }
};
template <bool Vec>
struct Inner<Fp16, Vec> {
  Raw8 v;
  __device__ __forceinline__ void load(const void *h, int64_t, int64_t at, int left) { v = load_raw8<true>(h, at, left); }
  __device__ __forceinline__ f4 times(s8 w, f4 acc) const {
    // instruction i takes value i of each lane's run: k = 8 q4 + i
#pragma unroll
    for (int i = 0; i < 8; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(Fp16::to((uint16_t)w[i]), __builtin_bit_cast(float, i < 4 ? v.lo[i] : v.hi[i - 4]), acc, 0, 0, 0);
    return acc;
  }
};

template <typename Tr, bool Vec>
__global__ __launch_bounds__(64 * kWaves) void few_down_kernel(FewArgs a) {
  constexpr int kPitch = 20;  // floats a row of s_o: 16 and a gap that keeps rows off each other's banks
  __shared__ __attribute__((aligned(16))) float s_o[(kFewPairs + kFewTokens) * kPitch];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;
  const int n0 = 16 * blockIdx.x, pairs = a.T * a.k;
  const int row = min(n0 + p16, a.d - 1);  // rows past the last repeat it
  const int used = a.plan->used, items = used + (a.f_sh > 0);
  for (int u = wave; u < items; u += kWaves) {
    const bool shared = u == used;
    const int f = shared ? a.f_sh : a.f, pitch = shared ? a.pitch_sh : a.pitch;
    const uint16_t *w = (shared ? a.sh_dn : a.dn + (int64_t)a.plan->expert[u] * a.d * a.f) + (int64_t)row * f;
    const void *h = shared ? a.h_sh : a.h;
    const int first = shared ? 0 : a.plan->start[u], rows = shared ? a.T : a.plan->start[u + 1] - first;
    const int64_t part = (int64_t)(shared ? a.T : pairs) * pitch;
    for (int r0 = 0; r0 < rows; r0 += 16) {
      const bool ok = r0 + p16 < rows;
      const int pair = !ok ? 0 : shared ? r0 + p16 : a.plan->pair[first + r0 + p16];
      f4 acc = {0.f, 0.f, 0.f, 0.f};
      constexpr int kDeep = 8;
      for (int k0 = 0; k0 < f; k0 += 32 * kDeep) {
        s8 wv[kDeep];
#pragma unroll
        for (int y = 0; y < kDeep; ++y) {
          const int k = k0 + 32 * y + 8 * q4;
          wv[y] = load_w<Vec>(w + k, f - k);
        }
#pragma unroll
        for (int y = 0; y < kDeep; ++y) {
          const int k = k0 + 32 * y + 8 * q4;
          Inner<Tr, Vec> hv;
          hv.load(h, part, (int64_t)pair * pitch + k, ok ? f - k : 0);
          acc = hv.times(wv[y], acc);
        }
      }
      if (ok) *reinterpret_cast<f4 *>(&s_o[((shared ? pairs : 0) + pair) * kPitch + 4 * q4]) = acc;
    }
  }
  __syncthreads();
  for (int i = tid; i < 16 * a.T; i += 64 * kWaves) {
    const int t = i >> 4, c = i & 15;
    if (n0 + c >= a.d) continue;
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) y += a.plan->gate[t * a.k + j] * s_o[(t * a.k + j) * kPitch + c];
    if (a.f_sh > 0) y += s_o[(pairs + t) * kPitch + c];
    if (a.y_f32) {
      if (a.add) y += static_cast<const float *>(a.add)[t * a.ld_add + n0 + c];
      static_cast<float *>(a.y)[t * a.ld_y + n0 + c] = y;
    } else {
      if (a.add) y += Tr::to(static_cast<const uint16_t *>(a.add)[t * a.ld_add + n0 + c]);
      static_cast<uint16_t *>(a.y)[t * a.ld_y + n0 + c] = Tr::from(y);
    }
  }
}

template <typename Tr, int VPL, bool Vec>
hipError_t few_of(const FewArgs &a, hipStream_t s) {
  const int64_t used = a.E < a.T * a.k ? a.E : a.T * a.k;
  const int64_t items = used * cdiv(a.f, 8) + cdiv(a.f_sh, 8);
  few_gate_up_kernel<Tr, VPL, Vec><<<dim3((unsigned)(items < 768 ? items : 768)), 64 * kWaves, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  few_down_kernel<Tr, Vec><<<dim3((unsigned)cdiv(a.d, 16)), 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}
template <typename Tr, int VPL>
hipError_t few_vec(const FewArgs &a, hipStream_t s) {
  const bool vec = a.d % 8 == 0 && a.f % 8 == 0 && a.f_sh % 8 == 0;
  return vec ? few_of<Tr, VPL, true>(a, s) : few_of<Tr, VPL, false>(a, s);
}
template <typename Tr>
hipError_t few_experts(const FewArgs &a, hipStream_t s) {
  if (a.E <= 64) return few_vec<Tr, 1>(a, s);
  if (a.E <= 128) return few_vec<Tr, 2>(a, s);
  if (a.E <= 256) return few_vec<Tr, 4>(a, s);
  if (a.E <= 512) return few_vec<Tr, 8>(a, s);
  return few_vec<Tr, 16>(a, s);
}

}  // namespace

hipError_t launch_few_layer(const FewArgs &a, bool fp16, hipStream_t s) {
  return fp16 ? few_experts<Fp16>(a, s) : few_experts<Bf16>(a, s);
}

}  // namespace moe
