// Device pieces shared by the 16-bit operators: element types with their
// matrix instruction, direct loads into LDS, and the search that maps a tile
// number to rows of a group.
#pragma once

#include "grouped_internal.h"

namespace moe {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  static __device__ __forceinline__ f4 mfma(s8 a, s8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  }
  // nearest, ties to even; NaN stays NaN
  static __device__ __forceinline__ uint16_t from(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
  static __device__ __forceinline__ float to(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
};
struct Fp16 {
  static __device__ __forceinline__ f4 mfma(s8 a, s8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint16_t from(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ __forceinline__ float to(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
};

// 16 bytes from each lane's own address to LDS: lane l's land at dst + 16 l.
// dst is the same for the whole wave.
__device__ __forceinline__ void load_lds16(const void *src, void *dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// Orders what a wave's lanes write to LDS before and read from it behind this
// point. The hardware runs a wave's LDS accesses in order; this keeps the compiler from
// moving them, or from running the lanes of a branch past it one side after the other.
__device__ __forceinline__ void wave_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// Lane p of each 16-lane group names four 16-bit elements of row p / 4 of a
// 4 x 16 block (columns 4 (p % 4) ..); it receives column p, rows 0..3.
__device__ __forceinline__ s4 read_lds_tr(const void *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)p);
}

// Workgroups go to the eight XCDs in turn, each with an L2 of its own. Of
// `total` work items, workgroup b takes the one that gives every XCD a run of
// consecutive items (so those that share operands share an L2), or -1 when it has none.
__device__ __forceinline__ int xcd_item(int b, int total) {
  const int run = (total + 7) >> 3;
  const int item = (b & 7) * run + (b >> 3);
  return (b >> 3) < run && item < total ? item : -1;
}
// Workgroups to launch for at most `most` items.
inline int64_t xcd_grid(int64_t most) { return (most + 7) / 8 * 8; }

struct GroupTile {
  int e;       // group, or -1: no such tile
  int first;   // first sorted row of the group
  int count;   // rows of the group
  int before;  // row tiles of the groups before it
  int total;   // row tiles of all groups
};

// Group that holds row tile m, when every group's rows are cut into tiles of
// `rows`. Every wave searches by itself: lane l adds up the tiles of its run
// of ceil(G / 64) groups, a prefix sum over the lanes finds the lane that
// holds tile m, and its run is walked again. Offsets outside [0, P] are
// taken as the nearest of the two and a group that ends before it begins as empty, so that no
// address formed from them leaves the caller's arrays. m is pick(total tiles),
// the same for the whole wave; with m < 0 only `total` is found.
template <typename Pick>
__device__ __forceinline__ GroupTile find_group(const int32_t *offsets, int G, int P, int rows, Pick pick) {
  const int lane = threadIdx.x & 63;
  const int run = (G + 63) >> 6;
  const int g0 = min(lane * run, G), g1 = min(g0 + run, G);
  auto at = [&](int g) { return min(max(offsets[g], 0), P); };
  int mine = 0;
  const int begin = at(g0);
  int prev = begin;
  for (int g = g0; g < g1; ++g) {
    const int next = at(g + 1);
    mine += (max(next - prev, 0) + rows - 1) / rows;
    prev = next;
  }
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(sum, d);
    if (lane >= d) sum += v;
  }
  GroupTile t;
  t.total = __builtin_amdgcn_readfirstlane(__shfl(sum, 63));
  const int m = pick(t.total);
  t.e = -1;
  t.first = t.count = t.before = 0;
  const uint64_t past = __ballot(sum > m);
  if (m < 0 || past == 0) return t;
  const int owner = __builtin_ctzll(past);
  int before = __shfl(sum - mine, owner);
  if (run == 1) {  // every lane holds one group: its bounds are in the lane
    t.e = owner;
    t.first = __builtin_amdgcn_readfirstlane(__shfl(begin, owner));
    t.count = __builtin_amdgcn_readfirstlane(__shfl(prev, owner)) - t.first;
    t.before = __builtin_amdgcn_readfirstlane(before);
    return t;
  }
  int g = __shfl(g0, owner);
  const int end = __shfl(g1, owner);
  int a = at(g);
  for (; g < end; ++g) {
    const int b = at(g + 1);
    const int n = (max(b - a, 0) + rows - 1) / rows;
    if (m < before + n) {
      t.e = g;
      t.first = a;
      t.count = b - a;
      t.before = before;
      break;
    }
    before += n;
    a = b;
  }
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.first = __builtin_amdgcn_readfirstlane(t.first);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  t.before = __builtin_amdgcn_readfirstlane(t.before);
  return t;
}

// Group number k in an order of roughly falling size: those of at least 3/2 of
// the average rows first, then of at least the average, of at least half of it, and the rest; ascending in each class.
// For work whose length goes by the group's rows: the longest starts first, so
// that the end is not one long piece. The lanes count their runs' groups of the four classes in 16
// bits each; one prefix sum serves all four.
__device__ __forceinline__ int group_by_size(const int32_t *offsets, int G, int P, int k) {
  const int lane = threadIdx.x & 63;
  const int run = (G + 63) >> 6;
  const int g0 = min(lane * run, G), g1 = min(g0 + run, G);
  auto at = [&](int g) { return min(max(offsets[g], 0), P); };
  const int64_t G2 = 2 * (int64_t)G, P2 = P;
  auto kind = [&](int n) {  // n against P / G
    const int64_t x = n * G2;
    return x >= 3 * P2 ? 0 : x >= 2 * P2 ? 1 : x >= P2 ? 2 : 3;
  };
  uint64_t mine = 0;
  int prev = at(g0);
  for (int g = g0; g < g1; ++g) {
    const int next = at(g + 1);
    mine += 1ull << (16 * kind(max(next - prev, 0)));
    prev = next;
  }
  uint64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t v = __shfl_up((unsigned long long)sum, d);
    if (lane >= d) sum += v;
  }
  const uint64_t all = __shfl((unsigned long long)sum, 63);
  int c = 0;
  for (; c < 3; ++c) {
    const int n = (int)(all >> (16 * c) & 0xffff);
    if (k < n) break;
    k -= n;
  }
  const int upto = (int)(sum >> (16 * c) & 0xffff);
  const uint64_t past = __ballot(upto > k);
  if (past == 0) return -1;
  const int owner = __builtin_ctzll(past);
  k -= __shfl(upto - (int)(mine >> (16 * c) & 0xffff), owner);  // which of the owner's
  int g = __shfl(g0, owner);
  for (int a = at(g);; ++g) {
    const int b = at(g + 1);
    if (kind(max(b - a, 0)) == c && k-- == 0) break;
    a = b;
  }
  return __builtin_amdgcn_readfirstlane(g);
}

}  // namespace moe
