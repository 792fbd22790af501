// Products grouped by expert with 16-bit operands, and their gradients, for
// gfx950.
//
//   forward          C[p][n]  = sum_k A[row(p)][k] W_e[n][k]
//   input gradient   dA[p][k] = sum_n dC[p][n] W_e[n][k]
//   weight gradient  dW_e[n][k] = sum_{p of e} dC[p][n] A[row(p)][k]
//
// All three are out[i][j] = sum_r L[i][r] R[j][r] with another dimension cut by
// the groups and another operand lying across r. Products are exact in fp32 and
// accumulate in fp32; the result is rounded once, to the output's type.
//
// Three kernels: few rows (bound by reading the weights), small tiles (bound by
// latency) and wide tiles (bound by the matrix instructions, or by the weights
// where groups are small). launch() chooses.

#include "grouped_device.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kBR = 64;  // r per step

// 16 bytes of zeros: what a lane reads in place of a unit outside the arrays.
__device__ const u4 g_zeros = {0u, 0u, 0u, 0u};

// A tile of `Rows` rows x 64 r, r contiguous (128 bytes a row, eight 16-byte
// units). Unit u of row i lies in slot u ^ ((i >> 1) & 7), so that the 16 rows
// of one matrix operand fetch fall on distinct banks.
__device__ __forceinline__ int straight_unit(int row, int slot) { return slot ^ ((row >> 1) & 7); }
// A tile of 64 r x 64 columns, columns contiguous. The 32-byte pair of units
// that one transposing fetch reads of a row is moved by the row, so that the four rows that
// 16 lanes fetch together fall on distinct banks.
__device__ __forceinline__ int across_unit(int row, int slot) { return slot ^ ((row & 3) << 1); }

// Forward: sorted row p takes no row of A. Its results are zeros whatever the
// weights hold (a product of zeros would pass on their infinities and NaN).
template <int Mode>
__device__ __forceinline__ bool masked_row(const GroupedArgs &a, int p) {
  if (Mode != kFwd) return false;
  const int at = a.a_row ? a.a_row[p] : p;
  return at < 0 || at >= a.a_rows;
}

// Four consecutive results from element `at` on, of which `left` exist.
template <typename Tr>
__device__ __forceinline__ void store4(const GroupedArgs &a, int64_t at, f4 v, int left, bool add) {
  if (a.out_f32) {
    float *o = static_cast<float *>(a.out) + at;
    if (a.vec_out) {
      if (add) v += *reinterpret_cast<const f4 *>(o);
      *reinterpret_cast<f4 *>(o) = v;
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x < left) o[x] = v[x] + (add ? o[x] : 0.f);
    }
  } else {
    uint16_t *o = static_cast<uint16_t *>(a.out) + at;
    if (a.vec_out) {
      *reinterpret_cast<u2 *>(o) = u2{(uint32_t)Tr::from(v[0]) | (uint32_t)Tr::from(v[1]) << 16,
                                      (uint32_t)Tr::from(v[2]) | (uint32_t)Tr::from(v[3]) << 16};
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x < left) o[x] = Tr::from(v[x]);
    }
  }
}

// Eight 16-bit elements at p, of which the first n exist. Rows that are not whole aligned
// units are read all the same 16 bytes at a time (global loads need no alignment), but
// for a row's last elements.
typedef u4 __attribute__((aligned(2))) u4_any;
template <bool Vec>
__device__ __forceinline__ u4 load_unit(const uint16_t *p, int n) {
  u4 v = {0u, 0u, 0u, 0u};
  if (Vec) {
    if (n > 0) v = *reinterpret_cast<const u4 *>(p);
  } else if (n >= 8) {
    v = *reinterpret_cast<const u4_any *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = i < n ? (uint32_t)p[i] : 0u;
      v[i >> 1] |= x << (16 * (i & 1));
    }
  }
  return v;
}

// ---------------------------------------------------------------- small tiles
// 64 x 64 outputs a workgroup of four waves, 64 r a step, any sizes and
// alignment. Operands are loaded into registers two steps ahead and go to the other LDS
// buffer behind the matrix instructions of the step before theirs. A call is a chain of
// nr / 64 steps of about 0.8 us: 1002 rows in 13 groups, 515 x 777, fp16, 12 us (one step ahead
// 17.5); 512 rows in 8 groups, 1024 x 1024, bf16, 9.6 us (12.8). For calls whose wide
// tiles would leave most CUs idle, and for operands the wide tiles cannot request.
constexpr int kSmall = 64;

template <typename Tr, int Mode, bool Vec>
__global__ __launch_bounds__(256) void grouped_small_kernel(GroupedArgs a) {
  constexpr int B = kSmall, U = B * 8 / 256;  // 16-byte units a thread stages of each operand and step
  constexpr bool kLAcross = Mode == kWgrad, kRAcross = Mode != kFwd;
  __shared__ __attribute__((aligned(16))) uint8_t s_l[2][B * kBR * 2];
  __shared__ __attribute__((aligned(16))) uint8_t s_r[2][B * kBR * 2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;

  // ---- which tile
  int e, first, count, i0, j0, ni, nj, nr;
  if (Mode == kWgrad) {
    const int tj = (a.K + B - 1) / B, ti = (a.N + B - 1) / B, per = ti * tj;
    e = blockIdx.x / per;
    if (e >= a.G) return;
    const int t = blockIdx.x - e * per;
    i0 = t / tj * B;
    j0 = (t - t / tj * tj) * B;
    first = min(max(a.offsets[e], 0), a.P);
    count = max(min(max(a.offsets[e + 1], 0), a.P) - first, 0);
    nr = count;
    ni = a.N - i0;
    nj = a.K - j0;
  } else {
    const int J = Mode == kFwd ? a.N : a.K, tj = (J + B - 1) / B;
    int item;
    const GroupTile g = find_group(a.offsets, a.G, a.P, B, [&](int total) {
      item = xcd_item(blockIdx.x, total * tj);
      return item < 0 ? -1 : item / tj;
    });
    if (g.e < 0) return;
    e = g.e;
    const int t = item - g.before * tj, mt = (g.count + B - 1) / B;
    const int jt = t / mt;
    i0 = (t - jt * mt) * B;
    j0 = jt * B;
    first = g.first;
    count = g.count;
    ni = count - i0;
    nj = J - j0;
    nr = Mode == kFwd ? a.K : a.N;
  }
  // (with no row of A at all nothing is read, and every result is that of a masked row)
  const int steps = Mode == kFwd && a.a_rows == 0 ? 0 : (nr + kBR - 1) / kBR;

  // ---- staging. Unit u = tid + 256 i: a straight operand's row u / 8, an
  // across operand's r = u / 8, eight r or columns at 8 (slot's unit). Straight rows past the
  // output's end repeat its last, and masked ones read some row that exists: their results are not
  // stored, or set to zero.
  const uint16_t *lp[U], *rp[U];  // at step 0; nullptr: zeros
  const uint16_t *L = Mode == kWgrad ? a.w : a.rows;
  const int64_t ldl = Mode == kWgrad ? a.ld_w : a.ld_rows;
  const uint16_t *R = Mode == kWgrad ? a.rows : a.w + (int64_t)e * a.N * a.K;
  const int64_t ldr = Mode == kWgrad ? a.ld_rows : a.ld_w;
  const int urow = tid >> 3;
  const int lslot = 8 * (kLAcross ? across_unit(urow, tid & 7) : straight_unit(urow, tid & 7));
  const int rslot = 8 * (kRAcross ? across_unit(urow, tid & 7) : straight_unit(urow, tid & 7));
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int row = urow + 32 * i;  // the slots' swap goes by bits that 32 i leaves alone
    if (kLAcross) {
      lp[i] = lslot < ni ? L + (int64_t)(first + row) * ldl + i0 + lslot : nullptr;
    } else {
      int64_t at = first + i0 + min(row, ni - 1);
      if (Mode == kFwd && a.a_row) at = a.a_row[at];
      if (Mode == kFwd) at = min(max(at, (int64_t)0), max((int64_t)a.a_rows - 1, (int64_t)0));
      lp[i] = L + at * ldl + lslot;
    }
    if (kRAcross) rp[i] = rslot < nj ? R + j0 + rslot + (Mode == kDgrad ? (int64_t)row * ldr : 0) : nullptr;
    else rp[i] = R + (int64_t)(j0 + min(row, nj - 1)) * ldr + rslot;
  }
  u4 lreg[2][U], rreg[2][U];
  auto load = [&](int s, u4 (&lreg)[U], u4 (&rreg)[U], auto whole) __attribute__((always_inline)) {  // whole: every r of the step exists
    constexpr bool kAll = decltype(whole)::value;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = s * kBR + urow + 32 * i;  // across operands: the unit's r
      if (Mode == kWgrad) {  // a masked row's dC may hold anything: both operands are zeros
        int at = -1;
        if (r < nr) at = a.a_row ? a.a_row[first + r] : first + r;
        const bool ok = at >= 0 && at < a.a_rows;
        lreg[i] = load_unit<Vec>(lp[i] + (int64_t)s * kBR * ldl, lp[i] && ok ? ni - lslot : 0);
        rreg[i] = load_unit<Vec>(rp[i] + (ok ? at * ldr : 0), rp[i] && ok ? nj - rslot : 0);
        continue;
      }
      lreg[i] = load_unit<Vec>(lp[i] + s * kBR, kAll ? 8 : nr - s * kBR - lslot);
      if (kRAcross) {
        rreg[i] = load_unit<Vec>(rp[i] + (int64_t)s * kBR * ldr, rp[i] && (kAll || r < nr) ? nj - rslot : 0);
      } else {
        rreg[i] = load_unit<Vec>(rp[i] + s * kBR, kAll ? 8 : nr - s * kBR - rslot);
      }
    }
  };
  auto keep = [&](int buf, const u4 (&lreg)[U], const u4 (&rreg)[U]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      *reinterpret_cast<u4 *>(s_l[buf] + 16 * (tid + 256 * i)) = lreg[i];
      *reinterpret_cast<u4 *>(s_r[buf] + 16 * (tid + 256 * i)) = rreg[i];
    }
  };

  const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
  f4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  auto fetch = [&](const uint8_t *t, int c0, int ks, bool across) {
    if (!across) return *reinterpret_cast<const s8 *>(t + (c0 + p16) * 128 + 16 * straight_unit(c0 + p16, 4 * ks + q4));
    s4 x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 32 * ks + 8 * q4 + 4 * h + (p16 >> 2), c = c0 + 4 * (p16 & 3);
      x[h] = read_lds_tr(t + row * 128 + 16 * across_unit(row, c >> 3) + 2 * (c & 7));
    }
    return s8{x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
  };
  constexpr std::false_type partly{};
  if (steps > 0) {
    load(0, lreg[0], rreg[0], partly);
    if (steps > 1) load(1, lreg[1], rreg[1], partly);
    keep(0, lreg[0], rreg[0]);
  }
  // step s out of LDS buffer `buf`; registers `buf` receive step s + 2, the others hold s + 1
  auto step = [&](int s, auto buf_, auto whole) __attribute__((always_inline)) {
    constexpr int buf = decltype(buf_)::value;
    __syncthreads();
    if (decltype(whole)::value || s + 2 < steps) load(s + 2, lreg[buf], rreg[buf], whole);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      s8 l[2], r[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] = fetch(s_l[buf], wi + 16 * i, ks, kLAcross);
        r[i] = fetch(s_r[buf], wj + 16 * i, ks, kRAcross);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = Tr::mfma(r[j], l[i], acc[i][j]);
    }
    if (decltype(whole)::value || s + 1 < steps) keep(buf ^ 1, lreg[buf ^ 1], rreg[buf ^ 1]);
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  int s = 0;
  for (; (s + 4) * kBR <= nr && s < steps; s += 2) {  // steps s + 2 and s + 3 are whole
    step(s, even, std::true_type{});
    step(s + 1, odd, std::true_type{});
  }
  for (; s < steps; s += 2) {
    step(s, even, partly);
    if (s + 1 < steps) step(s + 1, odd, partly);
  }

  // ---- results: lane holds output row p16 and four consecutive columns of each block
  const int64_t obase = Mode == kWgrad ? (int64_t)e * a.N * a.K : (int64_t)first * a.ld_out;
  const int64_t ldo = Mode == kWgrad ? a.K : a.ld_out;
  if (Mode == kWgrad && a.accumulate && count == 0) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = wi + 16 * i + p16;
    if (row >= ni) continue;
    const bool masked = masked_row<Mode>(a, first + i0 + row);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = wj + 16 * j + 4 * q4;
      if (col >= nj) continue;
      store4<Tr>(a, obase + (int64_t)(i0 + row) * ldo + j0 + col, masked ? f4{0.f, 0.f, 0.f, 0.f} : acc[i][j], nj - col, Mode == kWgrad && a.accumulate);
    }
  }
}

// ---------------------------------------------------------------- few rows
// Calls of a few rows read each touched group's weights once and are bound by
// that, so the weights are spread over all CUs: a workgroup takes up to 16 rows of
// a group and 32 output columns (forward) or 64 (input gradient); its eight waves share the sum
// and join in LDS, in order. Weights go straight from memory to operand registers.
// One token of 8 of 256 experts, 1024 x 2048 (34 MB of weights): 9.5 us, 3.5 TB/s; the rest is
// the launch, the search for the group and one trip to memory before the stream runs.
constexpr int kFewRows = 16;

template <typename Tr, int Mode>
__global__ __launch_bounds__(512) void grouped_few_kernel(GroupedArgs a) {
  constexpr int kCols = Mode == kFwd ? 32 : 64, NB = kCols / 16;  // 16-column blocks
  __shared__ __attribute__((aligned(16))) f4 s_part[8][Mode == kFwd ? 1 : NB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p16 = lane & 15, q4 = lane >> 4;
  const int J = Mode == kFwd ? a.N : a.K, nr = Mode == kFwd ? a.K : a.N;
  const int tj = (J + kCols - 1) / kCols;
  const GroupTile g = find_group(a.offsets, a.G, a.P, kFewRows, [&](int) { return (int)blockIdx.x / tj; });
  if (g.e < 0) return;
  const int t = blockIdx.x - g.before * tj, mt = (g.count + kFewRows - 1) / kFewRows;
  const int jt = t / mt, i0 = (t - jt * mt) * kFewRows, j0 = jt * kCols;
  const int ni = min(g.count - i0, kFewRows), nj = min(J - j0, kCols);
  int64_t at = g.first + i0 + p16;
  bool ok = p16 < ni;
  if (Mode == kFwd && a.a_row && ok) at = a.a_row[at];
  if (Mode == kFwd) ok = ok && at >= 0 && at < a.a_rows;
  const uint16_t *x = ok ? a.rows + at * a.ld_rows : nullptr;
  const uint16_t *W = a.w + (int64_t)g.e * a.N * a.K;
  const s8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  f4 acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};
  if constexpr (Mode == kFwd) {
    // wave: columns 16 (wave / 4) .., every fourth 32 of k
    const int n = j0 + 16 * (wave >> 2) + p16;
    const uint16_t *w = n < a.N ? W + (int64_t)n * a.K : nullptr;
    constexpr int kDeep = 8;
    for (int k0 = 32 * (wave & 3); k0 < nr; k0 += 128 * kDeep) {
      s8 wv[kDeep], xv[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int k = k0 + 128 * u + 8 * q4;
        wv[u] = w && k < nr ? *reinterpret_cast<const s8 *>(w + k) : zero;
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int k = k0 + 128 * u + 8 * q4;
        xv[u] = x && k < nr ? *reinterpret_cast<const s8 *>(x + k) : zero;
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) acc[0] = Tr::mfma(wv[u], xv[u], acc[0]);
    }
    s_part[wave][0][lane] = acc[0];
  } else {
    // wave: every eighth 32 of n. A lane reads four columns 4 p16 .. of rows n = 8 q4 .. + 7 and
    // hands the matrix instruction number c the eight values of column 4 p16 + c.
    const int col = 4 * p16;
    constexpr int kDeep = 2;
    for (int n0 = 32 * wave; n0 < nr; n0 += 256 * kDeep) {
      u2 wv[kDeep][8];
      s8 xv[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int n = n0 + 256 * u + 8 * q4;
#pragma unroll
        for (int y = 0; y < 8; ++y)
          wv[u][y] = n < nr && col < nj ? *reinterpret_cast<const u2 *>(W + (int64_t)(n + y) * a.K + j0 + col) : u2{0u, 0u};
        xv[u] = x && n < nr ? *reinterpret_cast<const s8 *>(x + n) : zero;
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          u4 v;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t lo = wv[u][2 * y][c >> 1], hi = wv[u][2 * y + 1][c >> 1];
            v[y] = c & 1 ? (lo >> 16) | (hi & 0xffff0000u) : (lo & 0xffffu) | (hi << 16);
          }
          acc[c] = Tr::mfma(__builtin_bit_cast(s8, v), xv[u], acc[c]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NB; ++c) s_part[wave][c][lane] = acc[c];
  }
  __syncthreads();
  // lane: row p16; forward: wave 0 and 1 take a 16-column block each, columns 4 q4 ..;
  // input gradient: block c's operand row m is column 4 m + c, so a lane has 4 (4 q4 + reg) + c
  if (Mode == kFwd) {
    if (wave < 2) {
      f4 v = s_part[4 * wave][0][lane];
#pragma unroll
      for (int y = 1; y < 4; ++y) v += s_part[4 * wave + y][0][lane];
      const int col = 16 * wave + 4 * q4;
      if (!ok) v = f4{0.f, 0.f, 0.f, 0.f};
      if (p16 < ni && col < nj) store4<Tr>(a, (int64_t)(g.first + i0 + p16) * a.ld_out + j0 + col, v, nj - col, false);
    }
  } else if (wave < 4) {  // wave: the four columns 4 (4 q4 + wave) ..
    f4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float sum = 0.f;
#pragma unroll
      for (int y = 0; y < 8; ++y) sum += reinterpret_cast<const float *>(&s_part[y][c][lane])[wave];
      v[c] = sum;
    }
    const int col = 4 * (4 * q4 + wave);
    if (p16 < ni && col < nj) store4<Tr>(a, (int64_t)(g.first + i0 + p16) * a.ld_out + j0 + col, v, nj - col, false);
  }
}

// ---------------------------------------------------------------- wide tiles
// 256 x 256 outputs a workgroup of eight waves (each 128 x 64: 128 accumulator
// registers a lane, two waves a SIMD), 64 r a step, two LDS buffers of a step's
// operands. Both halves (32 r) of a step pass through registers one half ahead
// of their use:
//   half 0: its matrix instructions, and the LDS reads of half 1;
//   meeting: the step's buffer is read out, the next step's has landed;
//   half 1: its matrix instructions, the LDS reads of the next step's half 0, and
//           the requests of the step after next into the buffer that is free.
// So a request has one whole step (2048 cycles of matrix instructions a SIMD) to land,
// and one meeting a step suffices.
//
// Output rows belong to the two row waves by alternating 16-row blocks, so
// that a tile of fewer rows (TI < 8) has work for both. Output columns are
// numbered so that a lane ends with 16 consecutive columns of a row in its four
// blocks: block j, operand row m holds column 16 (m / 4) + 4 j + m % 4 of the wave's 64.
//
// bf16, one group of 4096 rows, 4096 x 4096: forward 1400, input gradient 1375,
// weight gradient 1250 TFLOP/s (a library product of 8192^3 runs at 1470). Uneven groups of
// 8192 tokens: top-8 of 256 experts, 1024 x 2048, forward 380 us (720 TFLOP/s; 15 % of the matrix work
// is rows of padding, and the weights alone take 207 us at copy rate); top-2 of 16, 4096 x 2048, 281 us (980);
// weight gradient of top-8 of 64, 378 us (730).
constexpr int kTJ = 4;                  // 16 x 16 blocks of a wave along the columns
constexpr int kWide = 256;              // rows and columns of a tile
constexpr int kWideThreads = 512;
constexpr int kUnits = 4;               // requests of a thread for each operand of a step, 16 bytes each

// Where 1 KiB piece c (what one wave requests at once) of an operand lies in LDS.
// A straight operand's piece is eight rows of 128 bytes, whose 16-byte units are swapped
// by row so that the 16 rows of a fetch fall on distinct banks. An across
// operand's piece is r = c and r = c + 32, 512 bytes each, so that the four r that 16 lanes fetch
// together lie in four consecutive pieces. Gaps between the pieces keep those off each other's banks:
// 32 bytes a piece where a fetch takes 32 consecutive bytes of each r (the row operand), 16 and 128 bytes by
// the piece's last two bits where it takes four times 8 bytes at 32-byte steps (the column operand).
template <int Mode>
__device__ __forceinline__ constexpr int row_piece(int c) { return Mode == kWgrad ? c * 1056 : c * 1024; }
template <int Mode>
__device__ __forceinline__ constexpr int col_piece(int c) {
  return Mode == kFwd ? c * 1024 : c * 1024 + 16 * (c & 1) + 128 * ((c >> 1) & 1) + 256 * (c >> 2);
}
__device__ __forceinline__ int row_unit(int row, int slot) { return slot ^ ((row >> 1) & 7); }
__device__ __forceinline__ int col_unit(int row, int slot) { return slot ^ (((row >> 1) & 1) | ((row >> 4) & 3) << 1); }

// Keeps a wave's common address in scalar registers, apart from the lanes'
// offsets: left alone, the compiler holds their sums, two vector registers each.
__device__ __forceinline__ const char *uniform(const char *p) {
  asm("" : "+s"(p));
  return p;
}

struct WideTile {
  int e, first, count;  // group, its first row, its rows
  int i0, j0, ni, nj;   // the tile's first output row and column, and how many exist from there
  int nr;               // terms of the sum
};

template <typename Tr, int Mode, int TI, bool Gather, int Stages>
__device__ __forceinline__ void wide_body(const GroupedArgs &a, const WideTile t, uint8_t *s_l0, uint8_t *s_l1, uint8_t *s_l2,
                                          uint8_t *s_r0, uint8_t *s_r1, uint8_t *s_r2) {
  constexpr bool kLAcross = Mode == kWgrad, kRAcross = Mode != kFwd, kNear = Mode == kWgrad;
  constexpr int UL = kLAcross ? kUnits : (TI + 1) / 2;  // requests that hold rows of a tile of 32 TI
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave >> 2, wj = wave & 3;
  const int p16 = lane & 15, q4 = lane >> 4;
  const int steps = (t.nr + kBR - 1) / kBR;

  // ---- requests. Unit i is piece 8 i + wave: a straight operand's tile rows
  // 64 i + tid / 8, an across operand's r = 8 i + wave of the step in the lower 32 lanes and 32 more in the upper. Rows and
  // columns past the output's end repeat the last one; what they give is not stored.
  // Byte offsets are 32 bits from a base that is the same for the workgroup.
  const char *lbase, *rbase;
  uint32_t lv[kLAcross ? 1 : UL], rv[kRAcross ? 1 : kUnits];
  int lr, rr;  // this thread's r in a step: straight the first of its unit's eight, across that of unit 0
  const int col_wave = col_piece<Mode>(wave);  // adds to col_piece(8 i)
  if constexpr (kLAcross) {
    lr = wave + (lane & 32);
    lbase = (const char *)(a.w + (int64_t)t.first * a.ld_w + t.i0);
    lv[0] = (uint32_t)(lr * a.ld_w + min(8 * (tid & 31), t.ni - 8)) * 2;
  } else {
    const int row0 = tid >> 3;
    lr = 8 * row_unit(row0, tid & 7);
    constexpr bool gather = Mode == kFwd && Gather;
    const int64_t from = gather ? 0 : (int64_t)t.first + t.i0;
    const int64_t have = max((Mode == kFwd ? a.a_rows : a.P) - from, (int64_t)1);
    lbase = (const char *)(a.rows + min(from, (int64_t)(Mode == kFwd ? a.a_rows : a.P) - 1) * a.ld_rows);
#pragma unroll
    for (int i = 0; i < UL; ++i) {
      int row = min(row0 + 64 * i, t.ni - 1);
      if (gather) row = a.a_row[t.first + t.i0 + row];
      // a masked row reads some row that exists; its results are set to zero at the end
      row = (int)min(max((int64_t)row, (int64_t)0), have - 1);
      lv[i] = (uint32_t)(row * a.ld_rows + lr) * 2;
    }
  }
  if constexpr (kRAcross) {
    rr = wave + (lane & 32);
    const int col = min(8 * (tid & 31), t.nj - 8);
    if constexpr (Mode == kWgrad) {
      rbase = (const char *)(a.rows + t.j0);
      rv[0] = (uint32_t)col * 2;
    } else {
      rbase = (const char *)(a.w + (int64_t)t.e * a.N * a.K + t.j0);
      rv[0] = (uint32_t)(rr * a.ld_w + col) * 2;
    }
  } else {
    const int row0 = tid >> 3;
    rr = 8 * col_unit(row0, tid & 7);
    rbase = (const char *)(a.w + ((int64_t)t.e * a.N + t.j0) * a.K);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) rv[j] = (uint32_t)(min(row0 + 64 * j, t.nj - 1) * a.ld_w + rr) * 2;
  }
  int rrow[kUnits];  // weight gradient: the rows of A of the next requested step, -1: zeros (dC's rows are the same r)
  auto fetch_rows = [&](int s) __attribute__((always_inline)) {
    if constexpr (Mode == kWgrad) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int r = s * kBR + rr + 8 * i, p = t.first + min(r, t.nr - 1);
        const int at = Gather ? a.a_row[p] : p;
        rrow[i] = ((r < t.nr) & (at < a.a_rows)) ? at : -1;
      }
    }
  };
  // `s` is the step asked for, lbase and rbase stand at it; `whole`: every r of the step exists
  const int64_t lstep = kLAcross ? kBR * a.ld_w * 2 : kBR * 2, rstep = Mode == kDgrad ? kBR * a.ld_w * 2 : Mode == kFwd ? kBR * 2 : 0;
  auto request_l = [&](int s, int i, uint8_t *buf, auto whole) __attribute__((always_inline)) {
    const char *p = uniform(lbase + (kLAcross ? (lstep >> 3) * i : 0)) + lv[kLAcross ? 0 : i];
    if constexpr (Mode == kWgrad) p = rrow[i] >= 0 ? p : (const char *)&g_zeros;  // a masked row's dC may hold anything
    else if constexpr (!decltype(whole)::value) p = s * kBR + lr < t.nr ? p : (const char *)&g_zeros;
    load_lds16(p, buf + row_piece<Mode>(8 * i) + row_piece<Mode>(1) * wave);
  };
  auto request_r = [&](int s, int i, uint8_t *buf, auto whole) __attribute__((always_inline)) {
    const char *p;
    if constexpr (Mode == kWgrad) {
      p = rbase + (uint64_t)((uint32_t)rrow[i] * (uint32_t)(a.ld_rows * 2) + rv[0]);
      p = rrow[i] >= 0 ? p : (const char *)&g_zeros;
    } else {
      p = uniform(rbase + (kRAcross ? (rstep >> 3) * i : 0)) + rv[kRAcross ? 0 : i];
      if constexpr (!decltype(whole)::value) p = s * kBR + rr + (kRAcross ? 8 * i : 0) < t.nr ? p : (const char *)&g_zeros;
    }
    load_lds16(p, buf + col_piece<Mode>(8 * i) + col_wave);
  };

  // ---- operand fetches: half ks is r = 32 ks + 8 q4 .. + 7; of an across operand fetch h takes r = 32 ks + 8 q4 + 4 h + x.
  // Every address is a lane's part, kept in one register, and a constant: the constant
  // and the lane's part of a piece's number add up without carries into each other's gap bits.
  const int cl = 8 * q4 + (p16 >> 2);
  const int col_row = 16 * (p16 >> 2) + (p16 & 3);
  uint32_t lat[2], rat[2];  // of half 0 and 1 (across operands: the first serves both)
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    lat[ks] = kLAcross ? row_piece<Mode>(cl) + 32 * wi + 8 * (p16 & 3)
                       : (16 * wi + p16) * 128 + 16 * row_unit(p16, 4 * ks + q4);
    rat[ks] = kRAcross ? col_piece<Mode>(cl) + 128 * wj + 32 * (p16 & 3)
                       : (64 * wj + col_row) * 128 + 16 * col_unit(col_row, 4 * ks + q4);
    asm("" : "+v"(lat[ks]), "+v"(rat[ks]));
  }
  auto read_l = [&](const uint8_t *b, int i, int ks) __attribute__((always_inline)) {
    if constexpr (kLAcross) {
      const s4 x = read_lds_tr(b + lat[0] + 512 * ks + 64 * i), y = read_lds_tr(b + lat[0] + row_piece<Mode>(4) + 512 * ks + 64 * i);
      return s8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    } else {
      return *reinterpret_cast<const s8 *>(b + lat[ks] + 4096 * i);
    }
  };
  auto read_r = [&](const uint8_t *b, int j, int ks) __attribute__((always_inline)) {
    if constexpr (kRAcross) {
      const s4 x = read_lds_tr(b + rat[0] + 512 * ks + 8 * j), y = read_lds_tr(b + rat[0] + col_piece<Mode>(4) + 512 * ks + 8 * j);
      return s8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    } else {
      return *reinterpret_cast<const s8 *>(b + rat[ks] + 512 * j);
    }
  };

  f4 acc[TI][kTJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < kTJ; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  s8 l0[TI], r0[kTJ], l1[TI], r1[kTJ];

  // This wave's requests but the last `open` steps' have landed and its reads are done, and
  // everyone's behind the barrier.
  constexpr int kAsks = UL + kUnits;
  auto meet = [&](auto open) __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | decltype(open)::value * kAsks);  // vmcnt, lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  constexpr std::integral_constant<int, 0> none{};
  constexpr std::integral_constant<int, Stages - 2> ahead{};
  // One step out of buffers bl, br; nl, nr hold the next.
  auto step = [&](int s, uint8_t *bl, uint8_t *br, uint8_t *nl, uint8_t *nr, auto whole) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): half 0's operands, before half 1's are asked for
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      if (i == 0) {
#pragma unroll
        for (int j = 0; j < kTJ; ++j) r1[j] = read_r(br, j, 1);
      }
      l1[i] = read_l(bl, i, 1);
#pragma unroll
      for (int j = 0; j < kTJ; ++j) acc[i][j] = Tr::mfma(r0[j], l0[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    meet(ahead);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      constexpr int per = (kAsks + TI - 1) / TI;  // requests beside a row of blocks
#pragma unroll
      for (int y = i * per; y < (i + 1) * per; ++y) {
        if (y < UL) request_l(s + Stages, y, bl, whole);
        else if (y < kAsks) request_r(s + Stages, y - UL, br, whole);
      }
      if (i == 0) {
#pragma unroll
        for (int j = 0; j < kTJ; ++j) r0[j] = read_r(nr, j, 0);
      }
      l0[i] = read_l(nl, i, 0);
#pragma unroll
      for (int j = 0; j < kTJ; ++j) acc[i][j] = Tr::mfma(r1[j], l1[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    lbase += lstep;
    rbase += rstep;
  };
  // The weight gradient's variant of a step. Both its operands come from LDS
  // in pairs of 8-byte fetches, and a half held ahead spills; here the next
  // step is requested at the step's begin, operands are fetched one row of blocks ahead, and the meeting
  // stands at the end.
  auto step_near = [&](int s, uint8_t *bl, uint8_t *br, uint8_t *nl, uint8_t *nr, auto whole) __attribute__((always_inline)) {
    s8 l[2], r[2][kTJ];
#pragma unroll
    for (int j = 0; j < kTJ; ++j) r[0][j] = read_r(br, j, 0);
    l[0] = read_l(bl, 0, 0);
#pragma unroll
    for (int x = 0; x < 2 * TI; ++x) {
      const int ks = x / TI, i = x % TI;
      if (x < UL) request_l(s + 1, x, nl, whole);
      else if (x < UL + kUnits) request_r(s + 1, x - UL, nr, whole);
      if (x + 1 < 2 * TI) l[(x + 1) & 1] = read_l(bl, (x + 1) % TI, (x + 1) / TI);
      if (x == TI - 2) {
#pragma unroll
        for (int j = 0; j < kTJ; ++j) r[1][j] = read_r(br, j, 1);
      }
#pragma unroll
      for (int j = 0; j < kTJ; ++j) acc[i][j] = Tr::mfma(r[ks][j], l[x & 1], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    lbase += lstep;
    rbase += rstep;
    fetch_rows(s + 2);
    meet(none);
  };
  constexpr std::false_type partly{};
  if (steps > 0) {
    fetch_rows(0);
#pragma unroll
    for (int i = 0; i < UL; ++i) request_l(0, i, s_l0, partly);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) request_r(0, i, s_r0, partly);
    lbase += lstep;
    rbase += rstep;
    fetch_rows(1);
    if constexpr (kNear) {
      meet(none);
      int s = 0;
      for (; (s + 3) * kBR <= t.nr; s += 2) {  // steps s + 1 and s + 2 are whole
        step_near(s, s_l0, s_r0, s_l1, s_r1, std::true_type{});
        step_near(s + 1, s_l1, s_r1, s_l0, s_r0, std::true_type{});
      }
      for (; s < steps; s += 2) {  // an odd number of steps ends with one of zeros
        step_near(s, s_l0, s_r0, s_l1, s_r1, partly);
        step_near(s + 1, s_l1, s_r1, s_l0, s_r0, partly);
      }
    } else {
#pragma unroll
      for (int x = 1; x < Stages; ++x) {
#pragma unroll
        for (int i = 0; i < UL; ++i) request_l(x, i, x == 1 ? s_l1 : s_l2, partly);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) request_r(x, i, x == 1 ? s_r1 : s_r2, partly);
        lbase += lstep;
        rbase += rstep;
      }
      meet(std::integral_constant<int, Stages - 1>{});
#pragma unroll
      for (int j = 0; j < kTJ; ++j) r0[j] = read_r(s_r0, j, 0);
#pragma unroll
      for (int i = 0; i < TI; ++i) l0[i] = read_l(s_l0, i, 0);
      auto round = [&](int s, auto whole) __attribute__((always_inline)) {
        if constexpr (Stages == 2) {
          step(s, s_l0, s_r0, s_l1, s_r1, whole);
          step(s + 1, s_l1, s_r1, s_l0, s_r0, whole);
        } else {
          step(s, s_l0, s_r0, s_l1, s_r1, whole);
          step(s + 1, s_l1, s_r1, s_l2, s_r2, whole);
          step(s + 2, s_l2, s_r2, s_l0, s_r0, whole);
        }
      };
      int s = 0;
      for (; (s + 2 * Stages) * kBR <= t.nr; s += Stages) round(s, std::true_type{});  // the steps it asks for are whole
      for (; s < steps; s += Stages) round(s, partly);  // a part of a round ends with steps of zeros
    }
  }
  meet(none);  // the buffers are free

  // ---- results. A wave passes 16 rows of its columns at a time through 2 KiB of
  // LDS of its own, so that it stores whole 128-byte lines (from the accumulators' places it
  // would store 16 bytes of each line at once, which ran at 2.5 TB/s where lines run at
  // twice that). 16-byte unit u of row r lies in slot u ^ (r & 7).
  const int64_t obase = Mode == kWgrad ? (int64_t)t.e * a.N * a.K : (int64_t)t.first * a.ld_out;
  const int64_t ldo = Mode == kWgrad ? a.K : a.ld_out;
  if (Mode == kWgrad && a.accumulate && t.count == 0) return;
  uint8_t *mine = s_l0 + 2048 * wave;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int row0 = 16 * (wi + 2 * i);
    if (row0 >= t.ni) break;
    bool masked = false;
    if (Mode == kFwd) {
      int at = t.first + t.i0 + min(row0 + p16, t.ni - 1);
      if (Gather) at = a.a_row[at];
      masked = at < 0 || at >= a.a_rows;
    }
    f4 (&v)[kTJ] = acc[i];  // by reference: a copied row would be held as one vector of 16 through the loop, which spills
    if (masked) {
#pragma unroll
      for (int c = 0; c < kTJ; ++c) v[c] = f4{0.f, 0.f, 0.f, 0.f};
    }
    if (a.out_f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // columns 32 h ..: the lanes of two q4
        if (q4 >> 1 == h) {
#pragma unroll
          for (int c = 0; c < 4; ++c) *reinterpret_cast<f4 *>(mine + 128 * p16 + 16 * ((4 * (q4 & 1) + c) ^ (p16 & 7))) = v[c];
        }
        wave_sync();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = 8 * x + (lane >> 3), col = 64 * wj + 32 * h + 4 * (lane & 7);
          f4 w = *reinterpret_cast<const f4 *>(mine + 128 * r + 16 * ((lane & 7) ^ (r & 7)));
          if (row0 + r >= t.ni || col >= t.nj) continue;
          float *o = static_cast<float *>(a.out) + obase + (int64_t)(t.i0 + row0 + r) * ldo + t.j0 + col;
          if (a.vec_out && col + 4 <= t.nj) {
            if (Mode == kWgrad && a.accumulate) w += *reinterpret_cast<const f4 *>(o);
            *reinterpret_cast<f4 *>(o) = w;
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (col + y < t.nj) o[y] = w[y] + (Mode == kWgrad && a.accumulate ? o[y] : 0.f);
          }
        }
        wave_sync();
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        u4 w;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          w[x] = (uint32_t)Tr::from(v[c + (x >> 1)][2 * (x & 1)]) | (uint32_t)Tr::from(v[c + (x >> 1)][2 * (x & 1) + 1]) << 16;
        *reinterpret_cast<u4 *>(mine + 128 * p16 + 16 * ((2 * q4 + (c >> 1)) ^ (p16 & 7))) = w;
      }
      wave_sync();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * x + (lane >> 3), col = 64 * wj + 8 * (lane & 7);
        const s8 w = *reinterpret_cast<const s8 *>(mine + 128 * r + 16 * ((lane & 7) ^ (r & 7)));
        if (row0 + r >= t.ni || col >= t.nj) continue;
        uint16_t *o = static_cast<uint16_t *>(a.out) + obase + (int64_t)(t.i0 + row0 + r) * ldo + t.j0 + col;
        if (a.vec_out && col + 8 <= t.nj) {
          *reinterpret_cast<s8 *>(o) = w;
        } else {
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if (col + y < t.nj) o[y] = (uint16_t)w[y];
        }
      }
      wave_sync();
    }
  }
}

// Rows: of a tile, 256 or 128. Tiles of 128 rows leave LDS for a third buffer.
template <typename Tr, int Mode, bool Gather, int Rows>
__global__ __launch_bounds__(kWideThreads, 2) void grouped_wide_kernel(GroupedArgs a) {
  constexpr int kLBytes = row_piece<Mode>(Rows / 8), kRBytes = col_piece<Mode>(kWide / 8), Stages = Rows == 256 ? 2 : 3;
  // arrays of their own rather than one: the compiler then knows that reading one does not depend on a request into another
  __shared__ __attribute__((aligned(16))) uint8_t s_l0[kLBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s_l1[kLBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s_l2[Stages == 3 ? kLBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t s_r0[kRBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s_r1[kRBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s_r2[Stages == 3 ? kRBytes : 16];
  WideTile t;
  if constexpr (Mode == kWgrad) {
    const int tj = (a.K + kWide - 1) / kWide, ti = (a.N + kWide - 1) / kWide;
    const int per = ti * tj;
    const int k = blockIdx.x / per;
    if (k >= a.G) return;
    t.e = group_by_size(a.offsets, a.G, a.P, k);
    if (t.e < 0) return;
    const int x = blockIdx.x - k * per;
    t.i0 = x / tj * kWide;
    t.j0 = (x - x / tj * tj) * kWide;
    t.first = min(max(a.offsets[t.e], 0), a.P);
    t.count = max(min(max(a.offsets[t.e + 1], 0), a.P) - t.first, 0);
    t.nr = t.count;
    t.ni = a.N - t.i0;
    t.nj = a.K - t.j0;
    wide_body<Tr, Mode, 8, Gather, Stages>(a, t, s_l0, s_l1, s_l2, s_r0, s_r1, s_r2);
  } else {
    const int J = Mode == kFwd ? a.N : a.K;
    const int tj = (J + kWide - 1) / kWide;
    int item;
    const GroupTile g = find_group(a.offsets, a.G, a.P, Rows, [&](int total) {
      item = xcd_item(blockIdx.x, total * tj);
      return item < 0 ? -1 : item / tj;
    });
    if (g.e < 0) return;
    t.e = g.e;
    const int x = item - g.before * tj, mt = (g.count + Rows - 1) / Rows;
    const int jt = x / mt;
    t.i0 = (x - jt * mt) * Rows;
    t.j0 = jt * kWide;
    t.first = g.first;
    t.count = g.count;
    t.ni = t.count - t.i0;
    t.nj = J - t.j0;
    t.nr = Mode == kFwd ? a.K : a.N;
    if (Rows == 256 && t.ni > 128) wide_body<Tr, Mode, 8, Gather, Stages>(a, t, s_l0, s_l1, s_l2, s_r0, s_r1, s_r2);
    else if (t.ni > 64) wide_body<Tr, Mode, 4, Gather, Stages>(a, t, s_l0, s_l1, s_l2, s_r0, s_r1, s_r2);
    else wide_body<Tr, Mode, 2, Gather, Stages>(a, t, s_l0, s_l1, s_l2, s_r0, s_r1, s_r2);
  }
}

template <typename Tr, int Mode, int Rows>
hipError_t launch_wide(const GroupedArgs &a, hipStream_t s) {
  const int64_t used = a.G < a.P ? a.G : a.P;  // groups that can have rows
  const int64_t tiles = Mode == kWgrad ? (int64_t)a.G * cdiv(a.N, kWide) * cdiv(a.K, kWide)
                                       : (a.P + used * (Rows - 1)) / Rows * cdiv(Mode == kFwd ? a.N : a.K, kWide);
  const int64_t wgs = Mode == kWgrad ? tiles : xcd_grid(tiles);  // the weight gradient's kernel takes its tile by number
  if (!grid_fits(wgs, kWideThreads) || tiles >= INT32_MAX / 2) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs);
  if (Mode != kDgrad && a.a_row) grouped_wide_kernel<Tr, Mode, Mode != kDgrad, Rows><<<grid, kWideThreads, 0, s>>>(a);
  else grouped_wide_kernel<Tr, Mode, false, Rows><<<grid, kWideThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename Tr, int Mode, bool Vec>
hipError_t launch(const GroupedArgs &a, hipStream_t s) {
  const int64_t used = a.G < a.P ? a.G : a.P;  // groups that can have rows
  const int J = Mode == kFwd ? a.N : a.K;
  if constexpr (Vec) {
    const int64_t at_least = Mode == kWgrad ? (int64_t)a.G * cdiv(a.N, kWide) * cdiv(a.K, kWide)
                                            : (used > a.P / kWide ? used : a.P / kWide) * cdiv(J, kWide);
    // Wide tiles where at least half the CUs get one. Against small tiles, us, forward / input gradient / weight
    // gradient: 16 groups, 1024 rows, 1024 x 1024 (64, 64 and 256 wide tiles) 16.3 / 17.2 / 15.1 against 12.2 / 12.7 / 18.6;
    // 32 groups, 2048 rows (128, 128, 512) 21.0 / 23.4 / 26.5 against 24.7 / 24.7 / 32.6; 4 groups, 8192 rows (128, 128,
    // 64) 27.0 / 27.1 / 55.7 against 38.5 / 39.5 / 40.3; 8 groups, 1024 rows (32, 32, 128) 16.3 / 22.9 / 15.8 against 11.0 / 11.6 / 12.9.
    const bool wide = a.wide && at_least >= 128;
    if constexpr (Mode != kWgrad) {
      // Few rows whose weights are too few for wide tiles. Against small tiles at N = 1024, K = 2048, us, forward / input
      // gradient: 8 groups, 8 rows 9.4 / 9.0 against 13.2 / 10.5, 64 rows 11.6 / 9.0 against 13.6 / 11.2, 128 rows 18.6 / 11.6
      // against 13.7 / 11.4. Against wide ones: 64 rows of 256 groups 48 / 40 against 42 / 42.
      if (!wide && a.P <= 64) {
        const int64_t wgs = (a.P + used * (kFewRows - 1)) / kFewRows * cdiv(J, Mode == kFwd ? 32 : 64);
        if (!grid_fits(wgs, 512)) return hipErrorInvalidConfiguration;
        grouped_few_kernel<Tr, Mode><<<dim3((unsigned)wgs), 512, 0, s>>>(a);
        return hipGetLastError();
      }
    }
    if (wide) {
      // Tiles of 128 rows and three buffers where groups hold few rows, of 256 and two where they
      // hold many, by the average. Forward at 256 experts, N = 1024, K = 2048: 159 against 170 us at
      // 2 rows a group, 214 / 234 at 64, 380 / 385 at 256; 16 groups of 1024 rows: 301 / 284. Input gradient:
      // 162 / 171 at 2, 240 / 250 at 64, 305 / 288 at 128.
      if constexpr (Mode != kWgrad) {
        if (a.P < (int64_t)(Mode == kFwd ? 256 : 96) * a.G) return launch_wide<Tr, Mode, 128>(a, s);
      }
      return launch_wide<Tr, Mode, 256>(a, s);
    }
  }
  const int64_t tiles = Mode == kWgrad ? (int64_t)a.G * cdiv(a.N, kSmall) * cdiv(a.K, kSmall)
                                       : (a.P + used * (kSmall - 1)) / kSmall * cdiv(J, kSmall);
  if (!grid_fits(xcd_grid(tiles), 256)) return hipErrorInvalidConfiguration;
  grouped_small_kernel<Tr, Mode, Vec><<<dim3((unsigned)(Mode == kWgrad ? tiles : xcd_grid(tiles))), 256, 0, s>>>(a);
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
