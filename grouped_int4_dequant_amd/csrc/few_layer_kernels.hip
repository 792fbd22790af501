// A mixture-of-experts layer with 16-bit weights for a few tokens, for gfx950:
// two kernels.
//
//   ids, g = top-k of the logits     h[t][j] = silu(W_g x[t]) * (W_u x[t]) of expert ids[t][j]
//   y[t] = sum_j g[t][j] W_dn h[t][j] + shared + add[t]
//
// A decode batch has little use of each weight, so the bytes of the picked experts set the time.
//   gate/up  every workgroup repeats the top-k (a token a wave, or four) and sorts the pairs (token,
//            slot) by expert in LDS, in blocks of at most 16 pairs of one expert; the first one leaves that for
//            the second kernel. Then it walks over items of 8 columns of h of one block: 16 rows of W_gu,
//            eight of the gate and the eight that it multiplies. One to eight waves share an item's sum
//            and join in LDS, in order; the next item's weights are requested before that.
//   down     a workgroup owns 8 columns of y, its waves take one block after the other. A lane has eight
//            consecutive terms of the sum in 512, of all 8 columns and of up to four pairs, multiplied in fp32; the lanes'
//            sums are added up in a fixed order. What a block gives each of its pairs goes to LDS, and is added up there by
//            token in slot order. The matrix instructions have no part in it: with one or two pairs a block they would be
//            nearly empty, and laying h out for them took three times the loads of the weights (57 us at 16 tokens of 8
//            of 256 experts, 2048 x 512).
// One token of 8 of 256 experts and the shared one, 2048 x 512, bf16: 13.4 and 5.3 us for 38 and 19 MB; 16 tokens: 82 us for
// 426 MB and 52 for 214 (5.2 and 4.1 TB/s).
// Weights go straight from memory to registers. They are read once for each 16 pairs of an expert, but by down, where a row is longer
// than the 512 terms that a wave's lanes hold, again for each four (from L2).

#include "block_device.h"
#include "topk_device.h"

#include <type_traits>

namespace moe {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;   // of a gate/up workgroup
// Steps of weights asked for at once. One token's layer is a single round of items: everything is asked for at once there,
// but for unaligned rows, which are put together from single words and have no registers left for sixteen
// (283 spilled: 33.0 us against 13.4 at 8 of 256 experts, 1001 x 512).
constexpr int deep_of(bool one, bool vec) { return one && vec ? 16 : 8; }

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

// A barrier that leaves loads from memory in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

struct FewLds {
  uint64_t tokens[MOE_MAX_EXPERTS];  // of each expert, a bit a token (kFewTokens of them; a token picks an expert once)
  int32_t ids[kFewPairs];
  float gate[kFewPairs];
  int32_t expert[kFewPairs], first[kFewPairs], rows[kFewPairs], pair[kFewPairs];
  int32_t start[MOE_MAX_EXPERTS];    // each expert's first sorted pair
  int32_t blocks;
};

// Top-k of all tokens and the pairs sorted by expert, by one workgroup.
template <int VPL>
__device__ __forceinline__ void make_plan(const FewArgs &a, FewLds &s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pairs = a.T * a.k;
  for (int e = tid; e < a.E; e += 64 * kWaves) s.tokens[e] = 0;
  float v[VPL], next[VPL];
  // four tokens a wave, where a wave would have several (gate/up of 64 tokens, 8 of 64 experts, 1024 x 512: 48.0 -> 37.8 us; of
  // 50 tokens, 2 of 16, 1000 x 744: 17.3 -> 15.4; of 9 tokens, 16 of 64: 32.1 -> 29.9)
  const bool quarters = VPL == 1 && a.k <= 16 && a.T > kWaves;
  if constexpr (VPL == 1) {
    if (quarters)
      for (int t0 = 4 * wave; t0 < a.T; t0 += 4 * kWaves) {
        const int t = t0 + (lane >> 4), j = lane & 15;
        int id;
        float g;
        topk_quarter<4>(a.logits + (int64_t)min(t, a.T - 1) * a.E, a.E, a.k, lane, id, g);
        if (t < a.T && j < a.k) {
          s.ids[t * a.k + j] = id;
          s.gate[t * a.k + j] = g;
        }
      }
  }
  if (!quarters && wave < a.T) topk_load<VPL>(a.logits + (int64_t)wave * a.E, a.E, lane, next);
  for (int t = wave; !quarters && t < a.T; t += kWaves) {
    int id;
    float g;
#pragma unroll
    for (int r = 0; r < VPL; ++r) v[r] = next[r];
    if (t + kWaves < a.T) topk_load<VPL>(a.logits + (int64_t)(t + kWaves) * a.E, a.E, lane, next);
    topk_values<VPL>(v, a.E, a.k, lane, id, g);
    if (lane < a.k) {
      s.ids[t * a.k + lane] = id;
      s.gate[t * a.k + lane] = g;
    }
  }
  __syncthreads();
  // (kFewPairs is the number of threads)
  const int mine = tid < pairs ? s.ids[tid] : -1;
  const uint64_t bit = 1ull << (tid / a.k & 63);
  if (mine >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&s.tokens[mine]), (unsigned long long)bit);
  __syncthreads();
  if (wave == 0) {
    // lane l has the experts of its run: their blocks and pairs, then what lies before it
    const int run = (a.E + 63) >> 6, e0 = min(lane * run, a.E), e1 = min(e0 + run, a.E);
    int n = 0, p = 0;
    for (int e = e0; e < e1; ++e) {
      const int c = __popcll(s.tokens[e]);
      n += (c + 15) >> 4;
      p += c;
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
    if (lane == 63) s.blocks = ns;
    int b = ns - n, at = ps - p;
    for (int e = e0; e < e1; ++e) {
      s.start[e] = at;
      for (int left = __popcll(s.tokens[e]); left > 0; left -= 16) {
        s.expert[b] = e;
        s.first[b] = at;
        s.rows[b++] = min(left, 16);
        at += min(left, 16);
      }
    }
  }
  __syncthreads();
  // an expert's pairs by ascending token: every workgroup has to cut them into the same blocks
  if (mine >= 0) s.pair[s.start[mine] + __popcll(s.tokens[mine] & (bit - 1))] = tid;
  __syncthreads();
  if (blockIdx.x != 0) return;
  if (tid < pairs) {
    a.plan->pair[tid] = s.pair[tid];
    a.plan->gate[tid] = s.gate[tid];
    if (a.topk_ids) a.topk_ids[tid] = mine;
    if (a.topk_w) a.topk_w[tid] = s.gate[tid];
  }
  if (tid < s.blocks) {
    a.plan->expert[tid] = s.expert[tid];
    a.plan->first[tid] = s.first[tid];
    a.plan->rows[tid] = s.rows[tid];
  }
  if (tid == 0) a.plan->blocks = s.blocks;
}

// One token: its picks are the blocks. A workgroup needs the first `need` of them only, the one whose items are
// those of the last pick leaves all for the second kernel.
template <int VPL>
__device__ __forceinline__ void make_plan_one(const FewArgs &a, FewLds &s, int need, bool writer) {
  if (need > 0 && threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int id;
    float g;
    topk_wave<VPL>(a.logits, a.E, need, lane, id, g);
    if (lane < need) s.expert[lane] = id;
    if (writer && lane < a.k) {
      a.plan->expert[lane] = id;
      a.plan->gate[lane] = g;
      if (a.topk_ids) a.topk_ids[lane] = id;
      if (a.topk_w) a.topk_w[lane] = g;
    }
  }
  lds_barrier();
}

// Stores the first `left` of four inner values.
__device__ __forceinline__ void store_inner(float *q, f4 v, int left) {
  if (left >= 4) {
    *reinterpret_cast<f4 *>(q) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) q[i] = v[i];
  }
}

// One: a single token.
template <typename Tr, int VPL, bool Vec, bool One>
__global__ __launch_bounds__(64 * kWaves, 4) void few_gate_up_kernel(FewArgs a) {
  constexpr int kDeep = deep_of(One, Vec), kX = 8;
  __shared__ FewLds s;
  __shared__ __attribute__((aligned(16))) f4 s_part[2][kWaves][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;
  const int per = (a.f + 7) / 8, per_sh = (a.f_sh + 7) / 8;
  const int blocks_sh = a.f_sh > 0 ? (a.T + 15) / 16 : 0;
  const int items_sh = blocks_sh * per_sh;
  if constexpr (One) {
    // (every workgroup has one round of items here)
    const int last = min(((int)blockIdx.x + 1) * (kWaves >> a.share) - 1, items_sh + a.k * per - 1);
    make_plan_one<VPL>(a, s, last < items_sh ? 0 : (last - items_sh) / per + 1, last == items_sh + a.k * per - 1);
  } else {
    make_plan<VPL>(a, s);
  }
  const int items = items_sh + (One ? a.k : s.blocks) * per;
  // the waves of a workgroup take kWaves >> share items at a time; `sub` has n steps of 32 k of the sum, from kb on
  const int slots = kWaves >> a.share, slot = wave >> a.share, sub = wave & ((1 << a.share) - 1);
  const int n = (((a.d + 31) >> 5) + (1 << a.share) - 1) >> a.share;
  const int kb = 32 * n * sub + 8 * q4, kend = min(a.d, 32 * n * (sub + 1));

  struct Where {
    const uint16_t *w, *x;
    int c0, pair;  // first column; the lane's pair (token, if shared), -1: none
    bool shared;
  };
  auto locate = [&](int item) __attribute__((always_inline)) {
    Where t;
    t.shared = item < items_sh;  // the shared expert's items come first
    const int i = t.shared ? item : item - items_sh, each = t.shared ? per_sh : per;
    const int b = i / each, f = t.shared ? a.f_sh : a.f;
    t.c0 = 8 * (i - b * each);
    const bool ok = item < items;
    const uint16_t *W = t.shared ? a.sh_gu : a.gu + (int64_t)(ok ? s.expert[b] : 0) * 2 * a.f * a.d;
    t.w = W + (int64_t)(min(t.c0 + (p16 & 7), f - 1) + (p16 & 8 ? f : 0)) * a.d;  // columns past the last repeat it
    t.pair = -1;
    if (One) {
      if (p16 == 0 && ok) t.pair = t.shared ? 0 : b;
    } else if (t.shared) {
      if (16 * b + p16 < a.T) t.pair = 16 * b + p16;
    } else if (ok && p16 < s.rows[b]) {
      t.pair = s.pair[s.first[b] + p16];
    }
    t.x = a.x + (int64_t)(One || t.pair < 0 ? 0 : t.shared ? t.pair : t.pair / a.k) * a.ld_x;
    return t;
  };
  s8 wv[kDeep], xv[kX];
  auto request_x = [&](const Where &t, int y0) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < kX; ++y) {
      const int k = kb + 32 * (y0 + y);
      xv[y] = load_w<Vec>(t.x + k, t.pair >= 0 ? kend - k : 0);
    }
  };
  auto request = [&](const Where &t, int y0, int item) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < kDeep; ++y) {
      const int k = kb + 32 * (y0 + y);
      wv[y] = load_w<Vec>(t.w + k, item < items ? kend - k : 0);
    }
    request_x(t, y0);
  };
  const int rounds = (items + slots - 1) / slots;
  int buf = 0, round = blockIdx.x;
  if (round >= rounds) return;
  Where at = locate(round * slots + slot);
  request(at, 0, round * slots + slot);
  for (; round < rounds; round += gridDim.x) {
    const int item = round * slots + slot;
    f4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int y0 = 0; y0 < n; y0 += kDeep) {
      if (y0 > 0) request(at, y0, item);
#pragma unroll
      for (int h = 0; h < kDeep; h += kX) {
        if (h > 0) request_x(at, y0 + h);
#pragma unroll
        for (int y = 0; y < kX; ++y) acc = Tr::mfma(wv[h + y], xv[y], acc);
      }
    }
    const Where done = at;
    if (round + (int)gridDim.x < rounds) {
      at = locate(item + gridDim.x * slots);
      request(at, 0, item + gridDim.x * slots);
    }
    if (a.share > 0) {
      s_part[buf][wave][lane] = acc;
      lds_barrier();
      if (sub == 0) {
        acc = s_part[buf][wave][lane];
        for (int y = 1; y < 1 << a.share; ++y) acc += s_part[buf][wave + y][lane];
      }
      buf ^= 1;  // the next sums may be written while these are read; the barrier behind them ends both
    }
    if (sub == 0 && item < items) {
      // lane: pair p16; rows 4 q4 .. of the 16: columns 4 q4 .. of the gate, and behind them what it multiplies
      f4 h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = times_sigmoid(acc[i], acc[i]) * __shfl(acc[i], (lane + 32) & 63);
      const int c = done.c0 + 4 * q4, left = (done.shared ? a.f_sh : a.f) - c;
      if (done.pair >= 0 && q4 < 2 && left > 0) {
        if (done.shared) store_inner(a.h_sh + (int64_t)done.pair * a.pitch_sh + c, h, left);
        else store_inner(a.h + (int64_t)done.pair * a.pitch + c, h, left);
      }
    }
  }
}

// The sum of the values of four lanes 16 apart, in each of them.
__device__ __forceinline__ float sum_halves(float v) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);  // rows 0, 0, 2, 2 and 1, 1, 3, 3 of 16 lanes
  v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  const uint32_t y = __builtin_bit_cast(uint32_t, v);
  const auto q = __builtin_amdgcn_permlane32_swap(y, y, false, false);  // the lower half twice, and the upper
  return __builtin_bit_cast(float, (uint32_t)q[0]) + __builtin_bit_cast(float, (uint32_t)q[1]);
}

// Sums of eight values over the 64 lanes: lane l ends with those of values 2 (l % 4) and 2 (l % 4) + 1. Lanes that
// differ in the last two bits swap halves of what they hold first.
__device__ __forceinline__ void sum_lanes(const float (&v)[8], float &a, float &b) {
  const int lane = threadIdx.x & 63;
  const bool hi = lane & 2, odd = lane & 1;
  float w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = hi ? v[4 + i] : v[i], give = hi ? v[i] : v[4 + i];
    w[i] = keep + dpp_f32<0x4E>(give);  // lanes 2,3,0,1 of each four
  }
  a = (odd ? w[2] : w[0]) + dpp_f32<0xB1>(odd ? w[0] : w[2]);  // 1,0,3,2
  b = (odd ? w[3] : w[1]) + dpp_f32<0xB1>(odd ? w[1] : w[3]);
  a += dpp_f32<0x124>(a);  // four on, in each 16
  b += dpp_f32<0x124>(b);
  a += dpp_f32<0x128>(a);  // eight on
  b += dpp_f32<0x128>(b);
  a = sum_halves(a);
  b = sum_halves(b);
}

// As many waves as share the blocks evenly: up to 12 for one token, whose blocks are its picks, else 8, which leaves
// them registers for four pairs' values and sums beside the weights.
constexpr int down_waves(bool one) { return one ? 12 : 8; }
template <typename Tr, bool Vec, bool One>
__global__ __launch_bounds__(64 * down_waves(One)) void few_down_kernel(FewArgs a) {
  constexpr int kC = 8;             // columns of a workgroup
  constexpr int kR = One ? 1 : 4;   // pairs at a time (eight: 16 tokens' blocks 56 us against 51)
  constexpr int kSpan = 512;        // terms that a wave's lanes hold
  __shared__ __attribute__((aligned(16))) float s_o[(One ? 65 : kFewPairs + kFewTokens) * kC];
  __shared__ FewPlan s;  // what the first kernel left
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = kC * blockIdx.x, pairs = a.T * a.k;
  const int blocks_sh = a.f_sh > 0 ? (a.T + 15) / 16 : 0;
  int blocks;
  if constexpr (One) {
    blocks = a.k;
  } else {
    // all of it in one trip, whatever is in use
    for (int i = tid; i < pairs; i += blockDim.x) {
      s.expert[i] = a.plan->expert[i];
      s.first[i] = a.plan->first[i];
      s.rows[i] = a.plan->rows[i];
      s.pair[i] = a.plan->pair[i];
    }
    blocks = a.plan->blocks;
    lds_barrier();
  }
  for (int i = tid; i < pairs; i += blockDim.x) s.gate[i] = a.plan->gate[i];
  const int total = blocks + blocks_sh;

  struct Where {
    const uint16_t *w;
    int f, first, rows;  // terms of the sum; the block's first sorted pair (token, if shared), and how many
    bool shared;
  };
  auto locate = [&](int b) __attribute__((always_inline)) {
    Where t;
    t.shared = b < blocks_sh;  // the shared expert first
    b -= blocks_sh;
    t.f = t.shared ? a.f_sh : a.f;
    const int e = t.shared ? 0 : One ? a.plan->expert[b] : s.expert[b];
    t.w = (t.shared ? a.sh_dn : a.dn + (int64_t)__builtin_amdgcn_readfirstlane(e) * a.d * a.f) + (int64_t)n0 * t.f;
    t.first = t.shared ? 16 * (b + blocks_sh) : One ? b : __builtin_amdgcn_readfirstlane(s.first[b]);
    t.rows = One ? 1 : t.shared ? min(a.T - t.first, 16) : __builtin_amdgcn_readfirstlane(s.rows[b]);
    return t;
  };
  s8 wv[kC];
  auto request = [&](const Where &t, int k0) __attribute__((always_inline)) {
    const uint16_t *w = t.w + k0 + 8 * lane;
    const int left = t.f - k0 - 8 * lane;
#pragma unroll
    for (int c = 0; c < kC; ++c) wv[c] = load_w<Vec>(w + (int64_t)min(c, a.d - 1 - n0) * t.f, left);  // columns past the last repeat it
  };
  float acc[kR][kC];
  int pair[kR];
  // 512 terms of N pairs
  auto multiply = [&](const Where &t, int k0, auto n) __attribute__((always_inline)) {
    constexpr int N = decltype(n)::value;
    float hv[N][8];
    const float *h = (t.shared ? a.h_sh : a.h) + k0 + 8 * lane;
    const int left = t.f - k0 - 8 * lane, pitch = t.shared ? a.pitch_sh : a.pitch;
#pragma unroll
    for (int r = 0; r < N; ++r) widen8<Tr, true>(load_raw8<true, Vec>(h, (int64_t)pair[r] * pitch, left), hv[r]);
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = Tr::to((uint16_t)wv[c][i]);
#pragma unroll
        for (int r = 0; r < N; ++r) acc[r][c] = fmaf(w, hv[r][i], acc[r][c]);
      }
  };
  int b = wave;
  Where at{};
  if (b < total) {
    at = locate(b);
    request(at, 0);
  }
  while (b < total) {
    const Where t = at;
    for (int r0 = 0; r0 < t.rows; r0 += kR) {
      const int n = min(t.rows - r0, kR);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int q = t.first + r0 + min(r, n - 1);
        pair[r] = t.shared || One ? q : __builtin_amdgcn_readfirstlane(s.pair[q]);
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[r][c] = 0.f;
      }
      for (int k0 = 0; k0 < t.f; k0 += kSpan) {
        if (k0 > 0 || (r0 > 0 && t.f > kSpan)) request(t, k0);
        if (One || n == 1) multiply(t, k0, std::integral_constant<int, 1>{});
        else if (n == 2) multiply(t, k0, std::integral_constant<int, One ? 1 : 2>{});
        else multiply(t, k0, std::integral_constant<int, kR>{});
      }
      if (r0 + kR >= t.rows) {
        b += waves;
        if (b < total) {
          at = locate(b);
          request(at, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= n) break;
        float x, y;
        sum_lanes(acc[r], x, y);
        if (lane < 4) *reinterpret_cast<f2 *>(&s_o[((t.shared ? pairs : 0) + pair[r]) * kC + 2 * (2 * ((lane >> 1) & 1) + (lane & 1))]) = f2{x, y};
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < kC * a.T; i += blockDim.x) {
    const int t = i >> 3, c = i & 7;
    if (n0 + c >= a.d) continue;
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) y += s.gate[t * a.k + j] * s_o[(t * a.k + j) * kC + c];
    if (a.f_sh > 0) y += s_o[(pairs + t) * kC + c];
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
hipError_t few_of(FewArgs a, hipStream_t s) {
  const int64_t blocks_sh = a.f_sh > 0 ? cdiv(a.T, 16) : 0;
  // at most; one token's are its picks (a workgroup beyond the last item would write the plan once more)
  const int64_t pairs = (int64_t)a.T * a.k, blocks = a.T == 1 ? a.k : (a.E < pairs ? a.E : pairs) + pairs / 16;
  const int64_t items = blocks * cdiv(a.f, 8) + blocks_sh * cdiv(a.f_sh, 8);
  // a wave's part of a sum is what it asks for at once, where eight waves can make it so
  a.share = 0;
  while (a.share < 3 && ((a.d + 31) / 32 + (1 << a.share) - 1) >> a.share > deep_of(a.T == 1, Vec)) ++a.share;
  const int64_t rounds = cdiv(items, kWaves >> a.share);
  if (a.T == 1 && !grid_fits(rounds, 64 * kWaves)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(a.T == 1 || rounds < 512 ? rounds : 512));
  if (a.T == 1) few_gate_up_kernel<Tr, VPL, Vec, true><<<grid, 64 * kWaves, 0, s>>>(a);
  else few_gate_up_kernel<Tr, VPL, Vec, false><<<grid, 64 * kWaves, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n = blocks + blocks_sh, even = cdiv(n, cdiv(n, down_waves(a.T == 1))), waves = even < 4 ? 4 : even;
  const dim3 groups((unsigned)cdiv(a.d, 8));
  if (a.T == 1) few_down_kernel<Tr, Vec, true><<<groups, (unsigned)(64 * waves), 0, s>>>(a);
  else few_down_kernel<Tr, Vec, false><<<groups, (unsigned)(64 * waves), 0, s>>>(a);
  return hipGetLastError();
}
template <typename Tr, int VPL>
hipError_t few_vec(const FewArgs &a, hipStream_t s) {
  const bool vec = a.d % 8 == 0 && a.f % 8 == 0 && a.f_sh % 8 == 0;
  return vec ? few_of<Tr, VPL, true>(a, s) : few_of<Tr, VPL, false>(a, s);
}
template <typename Tr>
hipError_t few_experts(const FewArgs &a, hipStream_t s) {
  return a.E <= 64 ? few_vec<Tr, 1>(a, s) : a.E <= 256 ? few_vec<Tr, 4>(a, s) : few_vec<Tr, 16>(a, s);
}

}  // namespace

hipError_t launch_few_layer(const FewArgs &a, bool fp16, hipStream_t s) {
  return fp16 ? few_experts<Fp16>(a, s) : few_experts<Bf16>(a, s);
}

}  // namespace moe
