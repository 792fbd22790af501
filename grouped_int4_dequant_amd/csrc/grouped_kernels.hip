// Products grouped by expert with 16-bit operands, and their gradients, for
// gfx950.
//
//   forward          C[p][n]  = sum_k A[row(p)][k] W_e[n][k]
//   input gradient   dA[p][k] = sum_n dC[p][n] W_e[n][k]
//   weight gradient  dW_e[n][k] = sum_{p of e} dC[p][n] A[row(p)][k]
//
// All three are out[i][j] = sum_r L[i][r] R[j][r] with another dimension cut by
// the groups and another operand lying across r; one kernel body serves them.
// Products are exact in fp32 and accumulate in fp32; the result is rounded
// once, to the output's type.

#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kBR = 64;  // r per step

// 16 bytes of zeros: what a lane reads in place of a unit outside the arrays.
__device__ const u4 g_zeros = {0u, 0u, 0u, 0u};

// A tile of `Rows` rows x 64 r, r contiguous (128 bytes a row, eight 16-byte
// units). Unit u of row i lies in slot u ^ ((i >> 1) & 7), so that the 16 rows
// of one matrix operand fetch fall on distinct banks.
__device__ __forceinline__ int straight_unit(int row, int slot) { return slot ^ ((row >> 1) & 7); }
// A tile of 64 r x Cols columns, columns contiguous. The 32-byte pair of units
// that one transposing fetch reads of a row is moved by the row, so that the 16 rows of a
// fetch fall on distinct banks as far as the row length allows.
template <int Cols>
__device__ __forceinline__ int across_unit(int row, int slot) {
  return slot ^ (((((row & 3) | ((row >> 1) & 12))) & (Cols / 16 - 1)) << 1);
}

// Load `n` 16-bit elements one by one (operands whose rows are not whole aligned
// 16-byte units).
__device__ __forceinline__ u4 load_elems(const uint16_t *p, int64_t n) {
  u4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = i < n ? (uint32_t)p[i] : 0u;
    v[i >> 1] |= x << (16 * (i & 1));
  }
  return v;
}

template <typename Tr, int Mode, bool Vec, int BI, int BJ, int WI, int WJ>
__global__ __launch_bounds__(64 * WI * WJ) void grouped_kernel(GroupedArgs a) {
  constexpr int kThreads = 64 * WI * WJ;
  constexpr int TI = BI / WI / 16, TJ = BJ / WJ / 16;  // 16 x 16 blocks of a wave
  constexpr int UL = BI * 8 / kThreads, UR = BJ * 8 / kThreads;  // 16-byte units a thread stages per step
  static_assert(UL >= 1 && UR >= 1 && BI * 8 % kThreads == 0 && BJ * 8 % kThreads == 0, "whole units per thread");
  constexpr bool kLAcross = Mode == kWgrad, kRAcross = Mode != kFwd;
  __shared__ __attribute__((aligned(16))) uint8_t s_l[2][BI * kBR * 2];
  __shared__ __attribute__((aligned(16))) uint8_t s_r[2][BJ * kBR * 2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;

  // ---- which tile
  int e, first, count, i0, j0, ni, nj;  // ni, nj: rows and columns of the output that exist from i0, j0
  int nr;                               // length of the sum
  if (Mode == kWgrad) {
    const int tj = (a.K + BJ - 1) / BJ, ti = (a.N + BI - 1) / BI;
    const int per = ti * tj;
    e = blockIdx.x / per;
    const int t = blockIdx.x - e * per;
    i0 = t / tj * BI;
    j0 = (t - t / tj * tj) * BJ;
    first = min(max(a.offsets[e], 0), a.P);
    count = max(min(max(a.offsets[e + 1], 0), a.P) - first, 0);
    nr = count;
    ni = a.N - i0;
    nj = a.K - j0;
  } else {
    const int J = Mode == kFwd ? a.N : a.K;
    const int tj = (J + BJ - 1) / BJ;
    const int m = blockIdx.x / tj;
    const GroupTile g = find_group(a.offsets, a.G, a.P, BI, m);
    if (g.e < 0) return;
    e = g.e;
    const int t = blockIdx.x - g.before * tj, mt = (g.count + BI - 1) / BI;
    const int jt = t / mt;
    i0 = (t - jt * mt) * BI;
    j0 = jt * BJ;
    first = g.first;
    count = g.count;
    ni = count - i0;
    nj = J - j0;
    nr = Mode == kFwd ? a.K : a.N;
  }
  const int steps = (nr + kBR - 1) / kBR;

  // ---- what this thread stages: unit u = tid + kThreads i of each tile
  const uint16_t *lp[UL], *rp[UR];  // at step 0; nullptr: zeros at every step
  const uint16_t *L = Mode == kWgrad ? a.w : a.rows;
  const int64_t ldl = Mode == kWgrad ? a.ld_w : a.ld_rows;
  const uint16_t *R = Mode == kWgrad ? a.rows : a.w + (int64_t)e * a.N * a.K;
  const int64_t ldr = Mode == kWgrad ? a.ld_rows : a.ld_w;
  int lu[UL], ru[UR];  // straight: first r of the unit; across: its row r
#pragma unroll
  for (int i = 0; i < UL; ++i) {
    const int u = tid + kThreads * i;
    if (kLAcross) {
      constexpr int per = BI / 8;
      const int row = u / per, col = 8 * across_unit<BI>(row, u % per);
      lu[i] = row;
      lp[i] = col < ni ? L + (int64_t)(first + row) * ldl + i0 + col : nullptr;
    } else {
      const int row = u >> 3;
      lu[i] = 8 * straight_unit(row, u & 7);
      int64_t at = first + i0 + row;
      bool ok = row < ni;
      if (Mode == kFwd && a.a_row && ok) {
        at = a.a_row[at];
        ok = at >= 0 && at < a.a_rows;
      } else if (Mode == kFwd) {
        ok = ok && at < a.a_rows;
      }
      lp[i] = ok ? L + at * ldl + lu[i] : nullptr;
    }
  }
#pragma unroll
  for (int i = 0; i < UR; ++i) {
    const int u = tid + kThreads * i;
    if (kRAcross) {
      constexpr int per = BJ / 8;
      const int row = u / per, col = 8 * across_unit<BJ>(row, u % per);
      ru[i] = row;
      rp[i] = col < nj ? R + j0 + col + (Mode == kDgrad ? (int64_t)row * ldr : 0) : nullptr;
    } else {
      const int row = u >> 3;
      ru[i] = 8 * straight_unit(row, u & 7);
      rp[i] = row < nj ? R + (int64_t)(j0 + row) * ldr + ru[i] : nullptr;
    }
  }
  // rows of A that the weight gradient's next step gathers
  int rrow[UR];
  auto fetch_rows = [&](int s) {
    if (Mode != kWgrad) return;
#pragma unroll
    for (int i = 0; i < UR; ++i) {
      const int r = s * kBR + ru[i];
      int at = -1;
      if (r < nr) at = a.a_row ? a.a_row[first + r] : first + r;
      rrow[i] = at >= 0 && at < a.a_rows ? at : -1;
    }
  };
  auto stage = [&](int s, int buf) {
#pragma unroll
    for (int i = 0; i < UL; ++i) {
      const int r = s * kBR + lu[i];
      const uint16_t *p = lp[i];
      if (p) p += kLAcross ? (int64_t)s * kBR * ldl : s * kBR;
      const bool ok = p && r < nr;
      uint8_t *dst = s_l[buf] + 16 * (kThreads * i);
      if (Vec) {
        load_lds16(ok ? (const void *)p : (const void *)&g_zeros, dst + 1024 * wave);
      } else {
        const int left = kLAcross ? ni - 8 * across_unit<BI>(lu[i], (tid + kThreads * i) % (BI / 8)) : nr - r;
        *reinterpret_cast<u4 *>(dst + 16 * tid) = load_elems(p, ok ? left : 0);
      }
    }
#pragma unroll
    for (int i = 0; i < UR; ++i) {
      const int r = s * kBR + ru[i];
      const uint16_t *p = rp[i];
      bool ok = p && r < nr;
      if (Mode == kWgrad) {
        ok = p && rrow[i] >= 0;
        if (ok) p += (int64_t)rrow[i] * ldr;
      } else if (p) {
        p += kRAcross ? (int64_t)s * kBR * ldr : s * kBR;
      }
      uint8_t *dst = s_r[buf] + 16 * (kThreads * i);
      if (Vec) {
        load_lds16(ok ? (const void *)p : (const void *)&g_zeros, dst + 1024 * wave);
      } else {
        const int left = kRAcross ? nj - 8 * across_unit<BJ>(ru[i], (tid + kThreads * i) % (BJ / 8)) : nr - r;
        *reinterpret_cast<u4 *>(dst + 16 * tid) = load_elems(p, ok ? left : 0);
      }
    }
  };

  const int wi = wave / WJ * (BI / WI), wj = wave % WJ * (BJ / WJ);
  f4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

  // operand of 16 rows (or columns) from c0, r = 32 ks + 8 q4 ..+7
  auto straight = [&](const uint8_t *t, int c0, int ks) {
    const int row = c0 + p16;
    return *reinterpret_cast<const s8 *>(t + row * 128 + 16 * straight_unit(row, 4 * ks + q4));
  };
  auto across = [&](const uint8_t *t, int c0, int ks, auto cols) {
    constexpr int C = decltype(cols)::value;
    s8 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 32 * ks + 8 * q4 + 4 * h + (p16 >> 2);
      const int c = c0 + 4 * (p16 & 3);
      const s4 x = read_lds_tr(t + row * (2 * C) + 16 * across_unit<C>(row, c >> 3) + 2 * (c & 7));
      v[4 * h] = x[0]; v[4 * h + 1] = x[1]; v[4 * h + 2] = x[2]; v[4 * h + 3] = x[3];
    }
    return v;
  };

  if (steps > 0) {
    fetch_rows(0);
    stage(0, 0);
    fetch_rows(1);
  }
  for (int s = 0; s < steps; ++s) {
    const int buf = s & 1;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    s8 lf[2][TI], rf[2][TJ];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
        lf[ks][i] = kLAcross ? across(s_l[buf], wi + 16 * i, ks, std::integral_constant<int, BI>{}) : straight(s_l[buf], wi + 16 * i, ks);
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        rf[ks][j] = kRAcross ? across(s_r[buf], wj + 16 * j, ks, std::integral_constant<int, BJ>{}) : straight(s_r[buf], wj + 16 * j, ks);
    }
    if (s + 1 < steps) {
      stage(s + 1, buf ^ 1);
      fetch_rows(s + 2);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = Tr::mfma(rf[ks][j], lf[ks][i], acc[i][j]);
  }

  // ---- results: lane holds column p16 of block i (an output row) and four
  // consecutive output columns of block j
  const int64_t obase = Mode == kWgrad ? (int64_t)e * a.N * a.K : (int64_t)first * a.ld_out;
  const int64_t ldo = Mode == kWgrad ? a.K : a.ld_out;
  if (Mode == kWgrad && a.accumulate && count == 0) return;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int row = wi + 16 * i + p16;
    if (row >= ni) continue;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int col = wj + 16 * j + 4 * q4;
      if (col >= nj) continue;
      const int64_t at = obase + (int64_t)(i0 + row) * ldo + j0 + col;
      f4 v = acc[i][j];
      if (a.out_f32) {
        float *o = static_cast<float *>(a.out) + at;
        if (a.vec_out) {
          if (Mode == kWgrad && a.accumulate) v += *reinterpret_cast<const f4 *>(o);
          *reinterpret_cast<f4 *>(o) = v;
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (col + x < nj) o[x] = v[x] + (Mode == kWgrad && a.accumulate ? o[x] : 0.f);
        }
      } else {
        uint16_t *o = static_cast<uint16_t *>(a.out) + at;
        if (a.vec_out) {
          *reinterpret_cast<u2 *>(o) = u2{(uint32_t)Tr::from(v[0]) | (uint32_t)Tr::from(v[1]) << 16,
                                          (uint32_t)Tr::from(v[2]) | (uint32_t)Tr::from(v[3]) << 16};
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (col + x < nj) o[x] = Tr::from(v[x]);
        }
      }
    }
  }
}

template <typename Tr, int Mode, bool Vec>
hipError_t launch(const GroupedArgs &a, hipStream_t s) {
  constexpr int BI = 128, BJ = 128;
  int64_t tiles;
  if (Mode == kWgrad) {
    tiles = (int64_t)a.G * cdiv(a.N, BI) * cdiv(a.K, BJ);
  } else {
    const int64_t used = a.G < a.P ? a.G : a.P;  // groups that can have rows
    tiles = (a.P + used * (BI - 1)) / BI * cdiv(Mode == kFwd ? a.N : a.K, BJ);
  }
  if (!grid_fits(tiles, 256)) return hipErrorInvalidConfiguration;
  grouped_kernel<Tr, Mode, Vec, BI, BJ, 2, 2><<<dim3((unsigned)tiles), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename Tr, int Mode>
hipError_t launch_vec(const GroupedArgs &a, hipStream_t s) {
  return a.vec ? launch<Tr, Mode, true>(a, s) : launch<Tr, Mode, false>(a, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, GroupedMode mode, bool fp16, hipStream_t s) {
  switch (mode) {
    case kFwd: return fp16 ? launch_vec<Fp16, kFwd>(a, s) : launch_vec<Bf16, kFwd>(a, s);
    case kDgrad: return fp16 ? launch_vec<Fp16, kDgrad>(a, s) : launch_vec<Bf16, kDgrad>(a, s);
    default: return fp16 ? launch_vec<Fp16, kWgrad>(a, s) : launch_vec<Bf16, kWgrad>(a, s);
  }
}

}  // namespace moe
