// The norms before and after a block with its gate and residual, and their
// gradients, for gfx950.
//
//   p = o r(o) w_o      y = scale x + gate p      n = y r(y) w_n      r(v) = (mean v^2 + eps)^-1/2
//
//   gy  = dy + r(y) (w_n dn - yh mean(w_n dn yh))          yh = y r(y), oh = o r(o)
//   dx  = scale gy          dgate = sum_t gy p             dp = gate gy
//   d_o = r(o) (w_o dp - oh mean(w_o dp oh))    dw_o = sum_t dp oh    dw_n = sum_t dn yh
//
// Bound by memory: every row is read once into registers and everything that needs it
// is formed from there, in fp32; results are rounded once. n comes from y before y is
// rounded. Weights stay in registers (in the gradient in LDS) over the rows of a workgroup. bf16, 8192 rows of 2048
// with everything: 28.6 us for 134 MB (4.7 TB/s; a copy runs at 5.1), gradients 54 for 201 MB and 18 MB of column sums.
// The gradient has three workgroups a CU up to 2048 columns and one above; above 4096 its 1024 threads spill registers. 201 MB
// each: 4096 rows of 4096 61 us, 2048 of 8192 120, 1024 of 16384 345.

#include "block_device.h"

namespace moe {
namespace {

// A row is held by `W` waves, `V` runs of eight columns a lane; rows of fewer than
// four waves share a workgroup of four.
template <int W>
constexpr int threads_of() { return W < 4 ? 256 : 64 * W; }

// Sums over the waves of a row. The two halves of `buf` alternate from one sum to the next, so
// that one barrier a sum suffices. Every wave of the workgroup calls it.
template <int W>
struct RowSum {
  float *buf;  // [2][2][waves of the workgroup]
  int phase = 0;
  __device__ __forceinline__ void two(float &a, float &b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (W > 1) {
      constexpr int kWaves = threads_of<W>() / 64;
      const int wave = threadIdx.x >> 6;
      float *p = buf + 2 * kWaves * phase;
      phase ^= 1;
      if ((threadIdx.x & 63) == 0) {
        p[wave] = a;
        p[kWaves + wave] = b;
      }
      __syncthreads();
      const int first = wave / W * W;
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        a += p[first + i];
        b += p[kWaves + first + i];
      }
    }
  }
  __device__ __forceinline__ float one(float a) {
    float b = 0.f;
    two(a, b);
    return a;
  }
};

__device__ __forceinline__ float root(float squares, float inv_d, float eps) { return 1.f / sqrtf(squares * inv_d + eps); }

template <typename Tr, bool S32, bool Whole, int W, int V>
__global__ __launch_bounds__(threads_of<W>()) void norm_kernel(NormArgs a) {
  constexpr int kThreads = threads_of<W>(), G = kThreads / (64 * W);
  __shared__ float s_sum[4 * kThreads / 64];
  RowSum<W> sum{s_sum};
  const int g = threadIdx.x / (64 * W), tid = threadIdx.x - g * 64 * W;
  const float inv_d = 1.f / (float)a.d;
  int col[V], left[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = 8 * (tid + 64 * W * v);
    left[v] = a.d - col[v];
  }
  Raw8 o[V], x[V];
  auto load = [&](int row) __attribute__((always_inline)) {
    const bool ok = row < a.T;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (a.o) o[v] = load_raw8<false, Whole>(a.o, (int64_t)row * a.ld_o + col[v], ok ? left[v] : 0);
      if (a.x) x[v] = load_raw8<S32, Whole>(a.x, (int64_t)row * a.ld_x + col[v], ok ? left[v] : 0);
    }
  };
  int row = blockIdx.x * G + g;
  load(row);
  float wo[V][8], wn[V][8], gate[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (a.w_o) load8<Tr, Whole>(a.w_o, a.w_f32, col[v], left[v], wo[v]);
    if (a.n) load8<Tr, Whole>(a.w_n, a.w_f32, col[v], left[v], wn[v]);
  }
  int have = -1;  // row of gate in registers
  const int step = gridDim.x * G;
  for (int row0 = blockIdx.x * G; row0 < a.T; row0 += step, row += step) {
    float y[V][8];
    if (a.o) {
#pragma unroll
      for (int v = 0; v < V; ++v) widen8<Tr, false>(o[v], y[v]);
    }
    float xs[V][8];
    if (a.x) {
#pragma unroll
      for (int v = 0; v < V; ++v) widen8<Tr, S32>(x[v], xs[v]);
    }
    if (row0 + step < a.T) load(row + step);
    const bool ok = row < a.T;
    if (a.o) {
      if (a.gate && ok && row / a.period != have) {
        have = row / a.period;
#pragma unroll
        for (int v = 0; v < V; ++v) load8<Tr, Whole>(a.gate, a.w_f32, (int64_t)have * a.d + col[v], left[v], gate[v]);
      }
      if (a.w_o) {
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) sq += y[v][i] * y[v][i];
        const float r = root(sum.one(sq), inv_d, a.eps);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] = y[v][i] * r * wo[v][i];
      }
      if (a.gate) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] *= gate[v][i];
      }
    }
    if (a.x) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[v][i] = a.o ? fmaf(a.scale, xs[v][i], y[v][i]) : a.scale * xs[v][i];
    }
    if (a.y && ok) {
#pragma unroll
      for (int v = 0; v < V; ++v) store8<Tr, Whole>(a.y, S32, (int64_t)row * a.ld_y + col[v], left[v], y[v]);
    }
    if (a.n) {
      float sq = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) sq += left[v] > i ? y[v][i] * y[v][i] : 0.f;
      const float r = root(sum.one(sq), inv_d, a.eps);
      if (ok) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] = y[v][i] * r * wn[v][i];
          store8<Tr, Whole>(a.n, false, (int64_t)row * a.ld_n + col[v], left[v], y[v]);
        }
      }
    }
  }
}

// One chunk of rows for each group of W waves.
template <typename Tr, bool S32, bool Whole, int W, int V>
__global__ __launch_bounds__(threads_of<W>(), W == 16 ? 4 : 3) void norm_grad_kernel(NormGradArgs a) {
  constexpr int kThreads = threads_of<W>(), G = kThreads / (64 * W);
  __shared__ float s_sum[4 * kThreads / 64];
  // w_o, w_n and the gate as every lane uses them, in places of its own: they are read once a row, and leave
  // registers for three workgroups a CU
  constexpr bool kLds = 3 * V * 2 * 16 * kThreads <= 100 * 1024;
  __shared__ f4 s_w[kLds ? 3 * V * 2 * kThreads : 1];
  f4 own[kLds ? 1 : 3 * V * 2];
  auto put = [&](int what, int v, const float *f) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f4 x = {f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
      if constexpr (kLds) s_w[((what * V + v) * 2 + h) * kThreads + threadIdx.x] = x;
      else own[(what * V + v) * 2 + h] = x;
    }
  };
  auto get = [&](int what, int v, float *f) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f4 x;
      if constexpr (kLds) x = s_w[((what * V + v) * 2 + h) * kThreads + threadIdx.x];
      else x = own[(what * V + v) * 2 + h];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * h + i] = x[i];
    }
  };
  RowSum<W> sum{s_sum};
  const int g = threadIdx.x / (64 * W), tid = threadIdx.x - g * 64 * W;
  const int chunk = blockIdx.x * G + g;
  const float inv_d = 1.f / (float)a.d;
  int col[V], left[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = 8 * (tid + 64 * W * v);
    left[v] = a.d - col[v];
  }
  int begin, end;
  if (a.per_gate == 0) {
    begin = (int)min((int64_t)chunk * a.chunk_rows, (int64_t)a.T);
    end = (int)min((int64_t)begin + a.chunk_rows, (int64_t)a.T);
  } else {
    const int64_t b = chunk / a.per_gate, at = b * a.period + (int64_t)(chunk - b * a.per_gate) * a.chunk_rows;
    begin = (int)min(at, (int64_t)a.T);
    end = (int)min(min(at + a.chunk_rows, (b + 1) * a.period), (int64_t)a.T);
  }
  const bool live = chunk < a.chunks;
  if (!live) begin = end = 0;
  Raw8 o[V], y[V], dy[V], dn[V];
  auto load = [&](int row) __attribute__((always_inline)) {
    const bool ok = row < end;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int n = ok ? left[v] : 0;
      dy[v] = load_raw8<S32, Whole>(a.dy, (int64_t)row * a.ld_dy + col[v], a.dy ? n : 0);
      if (a.dn) {
        dn[v] = load_raw8<false, Whole>(a.dn, (int64_t)row * a.ld_dn + col[v], n);
        y[v] = load_raw8<S32, Whole>(a.y, (int64_t)row * a.ld_y + col[v], n);
      }
      if (a.o) o[v] = load_raw8<false, Whole>(a.o, (int64_t)row * a.ld_o + col[v], n);
    }
  };
  load(begin);
  float sum_o[V][8], sum_g[V][8], sum_n[V][8];
  float f8[8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (a.w_o) {
      load8<Tr, Whole>(a.w_o, a.w_f32, col[v], left[v], f8);
      put(0, v, f8);
    }
    if (a.dn) {
      load8<Tr, Whole>(a.w_n, a.w_f32, col[v], left[v], f8);
      put(1, v, f8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum_o[v][i] = sum_g[v][i] = sum_n[v][i] = 0.f;
  }
  int have = -1;
  // every group of the workgroup goes through as many rounds, for the barriers of the sums
  for (int round = 0; round < a.chunk_rows; ++round) {
    const int row = begin + round;
    const bool ok = row < end;
    if (G == 1 && !ok) break;
    float gy[V][8], of[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) widen8<Tr, S32>(dy[v], gy[v]);
    float yf[V][8], df[V][8];
    if (a.dn) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        widen8<Tr, S32>(y[v], yf[v]);
        widen8<Tr, false>(dn[v], df[v]);
      }
    }
    if (a.o) {
#pragma unroll
      for (int v = 0; v < V; ++v) widen8<Tr, false>(o[v], of[v]);
    }
    load(row + 1);
    float ro = 1.f, squares = 0.f;
    if (a.w_o) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) squares += of[v][i] * of[v][i];
    }
    if (a.dn) {
      float sq = 0.f, dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        get(1, v, f8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sq += yf[v][i] * yf[v][i];
          dot += yf[v][i] * f8[i] * df[v][i];
        }
      }
      sum.two(sq, dot);
      const float r = root(sq, inv_d, a.eps), along = dot * r * inv_d;
      if (ok) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          get(1, v, f8);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float hat = yf[v][i] * r;
            sum_n[v][i] += df[v][i] * hat;
            gy[v][i] += r * (f8[i] * df[v][i] - hat * along);
          }
        }
      }
    }
    if (a.dx && ok) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f8[i] = a.scale * gy[v][i];
        store8<Tr, Whole>(a.dx, S32, (int64_t)row * a.ld_dx + col[v], left[v], f8);
      }
    }
    if (!a.o) continue;
    if (a.gate && ok && row / a.period != have) {
      have = row / a.period;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        load8<Tr, Whole>(a.gate, a.w_f32, (int64_t)have * a.d + col[v], left[v], f8);
        put(2, v, f8);
      }
    }
    if (a.w_o) {
      // mean(w_o gate gy o), beside the squares
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float w8[8];
        get(0, v, w8);
        if (a.gate) get(2, v, f8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = w8[i] * gy[v][i] * (a.gate ? f8[i] : 1.f);  // w_o dp
          dot += left[v] > i ? t * of[v][i] : 0.f;
        }
      }
      sum.two(squares, dot);
      ro = root(squares, inv_d, a.eps);
      const float along = dot * ro * inv_d;
      if (ok) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float w8[8];
          get(0, v, w8);
          if (a.gate) get(2, v, f8);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float hat = of[v][i] * ro, dp = a.gate ? f8[i] * gy[v][i] : gy[v][i];
            sum_g[v][i] += gy[v][i] * hat * w8[i];
            sum_o[v][i] += dp * hat;
            of[v][i] = ro * (w8[i] * dp - hat * along);
          }
        }
      }
    } else if (ok) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.gate) get(2, v, f8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum_g[v][i] += gy[v][i] * of[v][i];
          of[v][i] = a.gate ? f8[i] * gy[v][i] : gy[v][i];
        }
      }
    }
    if (a.d_o && ok) {
#pragma unroll
      for (int v = 0; v < V; ++v) store8<Tr, Whole>(a.d_o, false, (int64_t)row * a.ld_do + col[v], left[v], of[v]);
    }
    if (a.dgate && a.per_gate == 0 && ok && (row + 1 == end || (row + 1) / a.period != have)) {  // the gate's last row
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t at = (int64_t)have * a.d + col[v];
        if (a.accumulate) {
          float f[8];
          load8<Tr, Whole>(a.dgate, a.g_f32, at, left[v], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum_g[v][i] += f[i];
        }
        store8<Tr, Whole>(a.dgate, a.g_f32, at, left[v], sum_g[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_g[v][i] = 0.f;
      }
    }
  }
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t at = (int64_t)chunk * a.pitch + col[v], kind = (int64_t)a.chunks * a.pitch;
    if (a.dw_o) store8<Tr, Whole>(a.part, true, at, left[v], sum_o[v]);
    if (a.dgate && a.per_gate) store8<Tr, Whole>(a.part, true, at + kind, left[v], sum_g[v]);
    if (a.dw_n) store8<Tr, Whole>(a.part, true, at + 2 * kind, left[v], sum_n[v]);
  }
}

// Adds up the chunks' column sums, in order: dw_o and dw_n over all chunks, a row of dgate
// over its own. A workgroup takes 64 columns of one result; sixteen waves share the chunks.
template <typename Tr>
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormGradArgs a, int first) {
  __shared__ float s_part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const int j = blockIdx.y + first;  // 0: dw_o, 1: dw_n, 2 ..: rows of dgate
  void *out = j == 0 ? a.dw_o : j == 1 ? a.dw_n : a.dgate;
  if (!out) return;
  const int64_t kind = j == 0 ? 0 : j == 1 ? 2 : 1;
  const float *p = a.part + kind * a.chunks * a.pitch + col;
  const int begin = j < 2 ? 0 : (j - 2) * a.per_gate, end = j < 2 ? a.chunks : begin + a.per_gate;
  float f = 0.f;
  if (col < a.d) {
    for (int c = begin + wave; c < end; c += 128) {
      float v[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        v[y] = 0.f;
        if (c + 16 * y < end) v[y] = p[(int64_t)(c + 16 * y) * a.pitch];
      }
#pragma unroll
      for (int y = 0; y < 8; ++y) f += v[y];
    }
  }
  s_part[wave][lane] = f;
  __syncthreads();
  if (wave != 0 || col >= a.d) return;
  f = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) f += s_part[w][lane];
  const int64_t at = (j < 2 ? 0 : (int64_t)(j - 2) * a.d) + col;
  if (a.g_f32) {
    float *q = static_cast<float *>(out) + at;
    *q = a.accumulate ? *q + f : f;
  } else {
    static_cast<uint16_t *>(out)[at] = Tr::from(f);
  }
}

template <typename Tr, bool S32, bool Whole, int W, int V>
hipError_t norm_at(const NormArgs &a, hipStream_t s) {
  constexpr int G = threads_of<W>() / (64 * W);
  // as many rows for every workgroup as 1024 workgroups of four waves need
  const int64_t wgs = cdiv(a.T, G), most = 1024 / (W < 4 ? 1 : W / 4);
  norm_kernel<Tr, S32, Whole, W, V><<<dim3((unsigned)cdiv(wgs, cdiv(wgs, most))), threads_of<W>(), 0, s>>>(a);
  return hipGetLastError();
}
template <typename Tr, bool S32, int W, int V>
hipError_t norm_of(const NormArgs &a, hipStream_t s) {
  return a.d % 8 == 0 ? norm_at<Tr, S32, true, W, V>(a, s) : norm_at<Tr, S32, false, W, V>(a, s);
}
template <typename Tr, bool S32>
hipError_t norm_by_width(const NormArgs &a, hipStream_t s) {
  if (a.d <= 512) return norm_of<Tr, S32, 1, 1>(a, s);
  if (a.d <= 1024) return norm_of<Tr, S32, 2, 1>(a, s);
  if (a.d <= 2048) return norm_of<Tr, S32, 4, 1>(a, s);
  if (a.d <= 4096) return norm_of<Tr, S32, 8, 1>(a, s);
  if (a.d <= 8192) return norm_of<Tr, S32, 16, 1>(a, s);
  return norm_of<Tr, S32, 16, 2>(a, s);
}

template <typename Tr, bool S32, bool Whole, int W, int V>
hipError_t grad_at(const NormGradArgs &a, hipStream_t s) {
  constexpr int G = threads_of<W>() / (64 * W);
  norm_grad_kernel<Tr, S32, Whole, W, V><<<dim3((unsigned)cdiv(a.chunks, G)), threads_of<W>(), 0, s>>>(a);
  return hipGetLastError();
}
template <typename Tr, bool S32, int W, int V>
hipError_t grad_of(const NormGradArgs &a, hipStream_t s) {
  return a.d % 8 == 0 ? grad_at<Tr, S32, true, W, V>(a, s) : grad_at<Tr, S32, false, W, V>(a, s);
}
template <typename Tr, bool S32>
hipError_t grad_by_width(const NormGradArgs &a, hipStream_t s) {
  if (a.d <= 512) return grad_of<Tr, S32, 1, 1>(a, s);
  if (a.d <= 1024) return grad_of<Tr, S32, 2, 1>(a, s);
  if (a.d <= 2048) return grad_of<Tr, S32, 4, 1>(a, s);
  if (a.d <= 4096) return grad_of<Tr, S32, 8, 1>(a, s);
  if (a.d <= 8192) return grad_of<Tr, S32, 16, 1>(a, s);
  return grad_of<Tr, S32, 16, 2>(a, s);
}
template <typename Tr>
hipError_t grad_all(const NormGradArgs &a, hipStream_t s) {
  if (a.T > 0) {
    const hipError_t e = a.stream_f32 ? grad_by_width<Tr, true>(a, s) : grad_by_width<Tr, false>(a, s);
    if (e != hipSuccess) return e;
  }
  // the results that are left: dw_o and dw_n, and the rows of dgate that chunks share
  const int rows_g = a.dgate && (a.per_gate || a.T == 0) ? a.gates : 0;
  const int first = a.dw_o ? 0 : a.dw_n ? 1 : 2;
  const int last = rows_g ? 2 + rows_g : a.dw_n ? 2 : a.dw_o ? 1 : 0;
  for (int y = first; y < last; y += 65535) {
    const int n = last - y < 65535 ? last - y : 65535;
    norm_columns_kernel<Tr><<<dim3((unsigned)cdiv(a.d, 64), (unsigned)n), 1024, 0, s>>>(a, y);
  }
  return hipGetLastError();
}

}  // namespace

NormChunks norm_chunks(int32_t T, int32_t period) {
  // about 768 chunks: three workgroups a CU at four waves a row
  int32_t rows = (int32_t)cdiv(T > 0 ? T : 1, 768);
  if (period <= rows) {
    rows = rows / period * period;
    return {rows, (int32_t)cdiv(T, rows), 0};
  }
  const int32_t per = (int32_t)cdiv(period, rows);
  return {rows, (int32_t)(cdiv(T, period) * per), per};
}

hipError_t launch_norm(const NormArgs &a, bool fp16, hipStream_t s) {
  if (fp16) return a.stream_f32 ? norm_by_width<Fp16, true>(a, s) : norm_by_width<Fp16, false>(a, s);
  return a.stream_f32 ? norm_by_width<Bf16, true>(a, s) : norm_by_width<Bf16, false>(a, s);
}

hipError_t launch_norm_grad(const NormGradArgs &a, bool fp16, hipStream_t s) {
  return fp16 ? grad_all<Fp16>(a, s) : grad_all<Bf16>(a, s);
}

}  // namespace moe
