// A mixture-of-experts layer with 16-bit weights for a few tokens, for gfx950:
// two kernels.
//
//   ids, g = top-k of the logits     h[t][j] = silu(W_g x[t]) * (W_u x[t]) of expert ids[t][j]
//   y[t] = sum_j g[t][j] W_dn h[t][j] + shared + add[t]
//
// A decode batch has little use of each weight, so the bytes of the picked experts set the time.
//   gate/up  every workgroup repeats the top-k (a token a wave) and sorts the pairs (token,
//            slot) by expert in LDS, in blocks of at most 16 pairs of one expert; the first one leaves that for
//            the second kernel. Then it walks over items of 8 columns of h of one block: 16 rows of W_gu,
//            eight of the gate and the eight that it multiplies. One to eight waves share an item's sum
//            and join in LDS, in order; the next item's weights are requested before that.
//   down     a workgroup owns 8 columns of y, its waves take one block after the other. The 16 operand
//            rows of a matrix instruction are the 8 columns over the first and the second half of the sum, against
//            up to eight pairs' halves, so that d / 8 workgroups fill the CUs. What a block gives each of its pairs
//            goes to LDS, and is added up there by token in slot order.
// Weights go straight from memory to operand registers and are read once (an expert of more than 16
// pairs again for each 16, from L2).

#include "block_device.h"
#include "topk_device.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kWaves = 8;   // of a gate/up workgroup
// Steps of weights asked for at once. One token's layer is a single round of items: everything is asked for at once there.
constexpr int deep_of(bool one) { return one ? 16 : 8; }

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
  if (wave < a.T) topk_load<VPL>(a.logits + (int64_t)wave * a.E, a.E, lane, next);
  for (int t = wave; t < a.T; t += kWaves) {
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

// An inner value as three bf16 parts that add up to it, each an array of its own: leading, middle and
// last eight bits, cut off rather than rounded, so that no rest changes its sign or leaves the range. Infinities and NaN
// are all in the first part.
__device__ __forceinline__ void store_inner(uint16_t *q, int64_t part, f4 v, int left) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= left) break;
    float rest = v[i];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t b = __builtin_bit_cast(uint32_t, rest);
      const bool finite = (b & 0x7f800000u) != 0x7f800000u;
      if (!finite && (b & 0x007fffffu)) b |= 0x00400000u;  // NaN stays NaN
      q[p * part + i] = (uint16_t)(b >> 16);
      rest = finite ? rest - __builtin_bit_cast(float, b & 0xffff0000u) : 0.f;
    }
  }
}

// One: a single token.
template <typename Tr, int VPL, bool Vec, bool One>
__global__ __launch_bounds__(64 * kWaves, 4) void few_gate_up_kernel(FewArgs a) {
  constexpr int kDeep = deep_of(One), kX = 8;
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
        if (done.shared) store_inner(a.h_sh + (int64_t)done.pair * a.pitch_sh + c, (int64_t)a.T * a.pitch_sh, h, left);
        else store_inner(a.h + (int64_t)done.pair * a.pitch + c, (int64_t)a.T * a.k * a.pitch, h, left);
      }
    }
  }
}

// Eight weights times a pair's eight inner values (their three parts), 32 terms a matrix instruction. bf16
// weights as they are; fp16 ones as two bf16 parts, of eight bits and of the three that are left.
template <typename Tr>
__device__ __forceinline__ f4 times_inner(const s8 (&w)[std::is_same_v<Tr, Fp16> ? 2 : 1], const s8 (&h)[3], f4 acc) {
#pragma unroll
  for (int p = 0; p < 3; ++p) acc = Bf16::mfma(w[0], h[p], acc);
  if constexpr (std::is_same_v<Tr, Fp16>) {
#pragma unroll
    for (int p = 0; p < 3; ++p) acc = Bf16::mfma(w[1], h[p], acc);
  }
  return acc;
}
template <typename Tr>
__device__ __forceinline__ void weight_parts(s8 w, s8 (&out)[std::is_same_v<Tr, Fp16> ? 2 : 1]) {
  if constexpr (std::is_same_v<Tr, Fp16>) {
    u4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = __builtin_bit_cast(uint32_t, Fp16::to((uint16_t)w[2 * i])), y = __builtin_bit_cast(uint32_t, Fp16::to((uint16_t)w[2 * i + 1]));
      hi[i] = (x >> 16) | (y & 0xffff0000u);
      const float rx = __builtin_bit_cast(float, x) - __builtin_bit_cast(float, x & 0xffff0000u);
      const float ry = __builtin_bit_cast(float, y) - __builtin_bit_cast(float, y & 0xffff0000u);
      lo[i] = (__builtin_bit_cast(uint32_t, rx) >> 16) | (__builtin_bit_cast(uint32_t, ry) & 0xffff0000u);
    }
    out[0] = __builtin_bit_cast(s8, hi);
    out[1] = __builtin_bit_cast(s8, lo);
  } else {
    out[0] = w;
  }
}

// As many waves as share the blocks evenly: up to 12 for one token, whose blocks are its picks, else 8, whose registers
// then hold both eights' inner values. 16 tokens of 8 of 256 experts, 2048 x 512: 57 us for 216 MB; 16 waves of half the registers
// 59, the next block's weights asked for a block ahead 53 (and 26 against 22 in fp16, which then spills).
constexpr int down_waves(bool one) { return one ? 12 : 8; }
template <typename Tr, bool Vec, bool One>
__global__ __launch_bounds__(64 * down_waves(One)) void few_down_kernel(FewArgs a) {
  constexpr int kPitch = 12;  // floats a row of s_o: 8 and a gap that keeps rows off each other's banks
  constexpr int kW = 16, kH = 4;  // steps of weights asked for at once, and of inner values
  constexpr int kX = One ? 1 : 2;  // eights of a block's pairs
  __shared__ __attribute__((aligned(16))) float s_o[(One ? 65 : kFewPairs + kFewTokens) * kPitch];
  __shared__ FewPlan s;  // what the first kernel left
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4, p8 = p16 & 7;
  const int n0 = 8 * blockIdx.x, pairs = a.T * a.k;
  const int row = min(n0 + p8, a.d - 1);  // rows past the last repeat it
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

  struct Where {
    const uint16_t *w, *h;
    int64_t part;
    int kb, kend, n;  // the lane's half of the sum, and its steps of 32
    int pitch, pair[kX], rows;  // the lane's pairs of the block's first and second eight
    bool shared;
  };
  auto locate = [&](int b) __attribute__((always_inline)) {
    Where t;
    t.shared = b < blocks_sh;  // the shared expert first
    b -= blocks_sh;
    const int f = t.shared ? a.f_sh : a.f, half = ((f + 63) >> 6) * 32;
    t.n = half >> 5;
    t.kb = (p16 & 8 ? half : 0) + 8 * q4;
    t.kend = p16 & 8 ? f : min(half, f);
    t.pitch = t.shared ? a.pitch_sh : a.pitch;
    t.h = t.shared ? a.h_sh : a.h;
    t.part = (int64_t)(t.shared ? a.T : pairs) * t.pitch;
    const int e = t.shared ? 0 : One ? a.plan->expert[b] : s.expert[b];
    t.w = (t.shared ? a.sh_dn : a.dn + (int64_t)e * a.d * a.f) + (int64_t)row * f;
    const int first = t.shared ? 16 * (b + blocks_sh) : One ? b : s.first[b];
    t.rows = One ? 1 : t.shared ? min(a.T - first, 16) : s.rows[b];
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      const int r = 8 * x + p8;
      t.pair[x] = r >= t.rows ? -1 : t.shared || One ? first + r : s.pair[first + r];
    }
    return t;
  };
  s8 wv[kW];
  auto request = [&](const Where &t, int y0) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < kW; ++y) {
      const int k = t.kb + 32 * (y0 + y);
      wv[y] = load_w<Vec>(t.w + k, t.kend - k);
    }
  };
  int b = wave;
  Where at{};
  if (b < blocks + blocks_sh) {
    at = locate(b);
    request(at, 0);
  }
  while (b < blocks + blocks_sh) {
    f4 acc[kX];
#pragma unroll
    for (int x = 0; x < kX; ++x) acc[x] = f4{0.f, 0.f, 0.f, 0.f};
    for (int y0 = 0; y0 < at.n; y0 += kW) {
      if (y0 > 0) request(at, y0);
#pragma unroll
      for (int g = 0; g < kW; g += kH) {
        if (y0 + g >= at.n) break;
        s8 hv[kX][kH][3];
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          if (8 * x >= at.rows) break;
          const uint16_t *h = at.h + (int64_t)max(at.pair[x], 0) * at.pitch;
#pragma unroll
          for (int y = 0; y < kH; ++y) {
            const int k = at.kb + 32 * (y0 + g + y);
#pragma unroll
            for (int p = 0; p < 3; ++p) hv[x][y][p] = load_w<Vec>(h + p * at.part + k, at.pair[x] >= 0 ? at.kend - k : 0);
          }
        }
#pragma unroll
        for (int y = 0; y < kH; ++y) {
          s8 parts[std::is_same_v<Tr, Fp16> ? 2 : 1];
          weight_parts<Tr>(wv[g + y], parts);
#pragma unroll
          for (int x = 0; x < kX; ++x) {
            if (8 * x >= at.rows) break;
            acc[x] = times_inner<Tr>(parts, hv[x][y], acc[x]);
          }
        }
      }
    }
    // lane: pair p16 % 8 and half p16 / 8 of the sum against rows 4 q4 .. of the 16; those of its own half count.
    // Where a sum is not finite, parts may have met that the values don't know (an infinite weight times a part
    // without bits): then it is formed once more, from whole values on the fp32 instruction.
    const bool counts = (p16 >> 3) == (q4 >> 1);
    const Where done = at;
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      if (8 * x >= done.rows) break;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) finite = finite && __builtin_fabsf(acc[x][i]) < __builtin_inff();
      if (__ballot(counts && !finite) == 0) continue;
      f4 again = {0.f, 0.f, 0.f, 0.f};
      const uint16_t *h = done.h + (int64_t)max(done.pair[x], 0) * done.pitch;
#pragma unroll 1
      for (int y = 0; y < done.n; ++y) {
        const int k = done.kb + 32 * y;
        const s8 w = load_w<Vec>(done.w + k, done.kend - k);
        s8 hv[3];
#pragma unroll
        for (int p = 0; p < 3; ++p) hv[p] = load_w<Vec>(h + p * done.part + k, done.pair[x] >= 0 ? done.kend - k : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // instruction i takes value i of each lane's run: k = 8 q4 + i
          const float v = (Bf16::to((uint16_t)hv[0][i]) + Bf16::to((uint16_t)hv[1][i])) + Bf16::to((uint16_t)hv[2][i]);
          again = __builtin_amdgcn_mfma_f32_16x16x4f32(Tr::to((uint16_t)w[i]), v, again, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[x][i] = __builtin_fabsf(acc[x][i]) < __builtin_inff() ? acc[x][i] : again[i];
    }
    b += waves;
    if (b < blocks + blocks_sh) {
      at = locate(b);
      request(at, 0);
    }
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      if (8 * x >= done.rows) break;
      f4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = acc[x][i] + __shfl(acc[x][i], (lane + 40) & 63);
      if (p16 < 8 && q4 < 2 && done.pair[x] >= 0)
        *reinterpret_cast<f4 *>(&s_o[((done.shared ? pairs : 0) + done.pair[x]) * kPitch + 4 * q4]) = v;
    }
  }
  __syncthreads();
  for (int i = tid; i < 8 * a.T; i += blockDim.x) {
    const int t = i >> 3, c = i & 7;
    if (n0 + c >= a.d) continue;
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) y += s.gate[t * a.k + j] * s_o[(t * a.k + j) * kPitch + c];
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
hipError_t few_of(FewArgs a, hipStream_t s) {
  const int64_t blocks_sh = a.f_sh > 0 ? cdiv(a.T, 16) : 0;
  const int64_t pairs = (int64_t)a.T * a.k, blocks = (a.E < pairs ? a.E : pairs) + pairs / 16;  // at most
  const int64_t items = blocks * cdiv(a.f, 8) + blocks_sh * cdiv(a.f_sh, 8);
  // a wave's part of a sum is what it asks for at once, where eight waves can make it so
  a.share = 0;
  while (a.share < 3 && ((a.d + 31) / 32 + (1 << a.share) - 1) >> a.share > deep_of(a.T == 1)) ++a.share;
  const int64_t rounds = cdiv(items, kWaves >> a.share);
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
