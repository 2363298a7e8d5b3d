// Root-mean-square norm of the residual stream on gfx950, forward and backward.
//
//   s = x + residual          (rounded to the inputs' type: the stream that the next layer adds to)
//   y = s r w,  r = (mean s^2 + eps)^(-1/2)
// and, for the products in 8 bits behind it, y as e4m3 with one scale a token:
//   scale = max |y| / 448,  q = round(y / scale).
// Backward, with v = s r:  dx = ds + r (w dy - v mean(w dy v)),  dw = sum over tokens of dy v.
//
// The norm is of the stream as it is stored, so that the backward pass, which has nothing else,
// differentiates what the forward computed.
//
// Bound: HBM, every array once.  A row is one wave's (up to 8 times 16 bytes a lane; its sums need no
// LDS), or for wider rows a workgroup's of 4 waves.  Measured, 16387 x 2048 bf16: forward with residual 46 us (268 MB
// at 5.8 TB/s, part of it still in the last-level cache), backward 57 us (268 MB at 4.7) and 5 us to add the weight's
// gradient; 64 x 2048 to 8 bits 4.8 us.
#include <type_traits>

#include "block_kernels.h"
#include "row_io.h"

namespace falcon {
namespace {

constexpr int THR = 256;
constexpr float F8_MAX = 448.f;      // the largest e4m3 number
constexpr float LEAST = 1e-30f;      // rows of zeros are scaled as if this were their largest entry

// The sum (largest) over the W waves of a row; `turn` makes consecutive calls use different places.
template <int W> __device__ __forceinline__ float row_sum(float x, float (*part)[4], int turn) {
  x = wave_sum(x);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = x;
    __syncthreads();
    x = (part[turn][0] + part[turn][1]) + (part[turn][2] + part[turn][3]);
  }
  return x;
}
template <int W> __device__ __forceinline__ unsigned row_max(unsigned x, float (*part)[4], int turn) {
  x = wave_max(x);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = __uint_as_float(x);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) x = max(x, __float_as_uint(part[turn][i]));
  }
  return x;
}

template <int E> __device__ __forceinline__ void load_weight(const float *w, int at, float (&o)[E]) {
  if (w) { load_f32<E>(w + at, o); return; }
#pragma unroll
  for (int j = 0; j < E; ++j) o[j] = 1.f;
}

// e4m3, to nearest even
__device__ __forceinline__ unsigned f8x4(float a, float b, float c, float d) {
  int v = 0;
  v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, v, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (unsigned)v;
}
__device__ __forceinline__ void store_f8(unsigned char *p, const float (&v)[8]) {
  *reinterpret_cast<uint2 *>(p) = uint2{f8x4(v[0], v[1], v[2], v[3]), f8x4(v[4], v[5], v[6], v[7])};
}
__device__ __forceinline__ void store_f8(unsigned char *p, const float (&v)[4]) {
  *reinterpret_cast<unsigned *>(p) = f8x4(v[0], v[1], v[2], v[3]);
}

// y / scale, the nearest fp32 number: by a rounded reciprocal alone, ties of the 8-bit rounding would go to either side.
// With scale = m 2^e, y 2^-e is exact, and two corrections by the remainder of y 2^-e after q m give the quotient to the last
// bit (Markstein's theorem: q is within a step after the first), in 6 instructions.  16387 x 768 bf16: 18.9 us, 20.1 with a
// division an entry (17.7 by the reciprocal); 16384 x 4096 112.7 both (110.4).
struct RowScale {
  float m, inv, down;      // mantissa, its reciprocal, 2^-e; an infinite scale leaves zeros, and a NaN NaN
  __device__ __forceinline__ explicit RowScale(float scale) {
    const unsigned u = __float_as_uint(scale), e = u & 0x7f800000u;
    m = __uint_as_float((u & 0x007fffffu) | 0x3f800000u);
    inv = 1.f / m;
    down = e < 0x7f800000u ? __uint_as_float(0x7f000000u - e) : 1.f / scale;
  }
  __device__ __forceinline__ float divide(float y) const {
    y *= down;
    float q = y * inv;
    q = fmaf(fmaf(-q, m, y), inv, q);
    return fmaf(fmaf(-q, m, y), inv, q);
  }
};

// W waves a row, V times 16 bytes a lane.
template <typename T, int W, int V, bool Q8> __global__ __launch_bounds__(THR) void norm_fwd(NormArgs a) {
  constexpr int E = PER16<T>, ROWS = 4 / W;
  __shared__ float part[4][4];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x, D = a.width;
  const int row0 = W == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  for (int row = row0, k = 0; row < a.tokens; row += gridDim.x * ROWS, k ^= 2) {
    const size_t base = (size_t)row * D;
    u4 raw[V], add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * W * 64 + lane) * E;
      raw[i] = c < D ? load16(static_cast<const T *>(a.x) + base + c) : u4{0, 0, 0, 0};
      if (a.residual) add[i] = c < D ? load16(static_cast<const T *>(a.residual) + base + c) : u4{0, 0, 0, 0};
    }
    float ss = 0.f;
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * W * 64 + lane) * E;
        float p[E], q[E];
        widen(raw[i], p);
        widen(add[i], q);
#pragma unroll
        for (int j = 0; j < E; ++j) p[j] += q[j];
        raw[i] = narrow(p);
        if (a.s && c < D) store16(static_cast<T *>(a.s) + base + c, raw[i]);
      }
    }
    float r = 1.f;
    if (a.norm) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float p[E];
        widen(raw[i], p);
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(p[j], p[j], ss);
      }
      r = rsqrtf(row_sum<W>(ss, part, k) * a.inv_width + a.eps);
    }
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * W * 64 + lane) * E;
        if (c >= D) continue;
        float p[E], w[E];
        widen(raw[i], p);
        load_weight<E>(a.w, c, w);
#pragma unroll
        for (int j = 0; j < E; ++j) p[j] = p[j] * r * w[j];
        store16(static_cast<T *>(a.y) + base + c, narrow(p));
      }
    } else {
      float y[V][E];
      unsigned top = 0;        // of the absolute values' bits: a NaN is larger than every number
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * W * 64 + lane) * E;
        float w[E];
        widen(raw[i], y[i]);
        if (c < D) load_weight<E>(a.w, c, w);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          y[i][j] = c < D ? y[i][j] * r * w[j] : 0.f;
          top = max(top, __float_as_uint(y[i][j]) & 0x7fffffffu);
        }
      }
      top = max(row_max<W>(top, part, k + 1), __float_as_uint(LEAST));
      const float scale = __uint_as_float(top) / F8_MAX;
      const RowScale by(scale);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * W * 64 + lane) * E;
        if (c >= D) continue;
#pragma unroll
        for (int j = 0; j < E; ++j) y[i][j] = by.divide(y[i][j]);
        store_f8(static_cast<unsigned char *>(a.y) + base + c, y[i]);
      }
      if (lane == 0) a.scale[row] = scale;
    }
  }
}

template <typename T, int W, int V> __global__ __launch_bounds__(THR) void norm_bwd(NormArgs a) {
  constexpr int E = PER16<T>, ROWS = 4 / W;
  __shared__ float part[4][4];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x, D = a.width;
  const int row0 = W == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  float dw[V][E] = {};
  for (int row = row0, k = 0; row < a.tokens; row += gridDim.x * ROWS, k ^= 2) {
    const size_t base = (size_t)row * D;
    u4 sv[V], gv[V], hv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * W * 64 + lane) * E;
      const bool on = c < D;
      sv[i] = on ? load16(static_cast<const T *>(a.x) + base + c) : u4{0, 0, 0, 0};
      gv[i] = on ? load16(static_cast<const T *>(a.dy) + base + c) : u4{0, 0, 0, 0};
      hv[i] = on && a.ds ? load16(static_cast<const T *>(a.ds) + base + c) : u4{0, 0, 0, 0};
    }
    float ss = 0.f, inner = 0.f;       // sums of s^2 and of w dy s
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * W * 64 + lane) * E;
      float s[E], g[E], w[E];
      widen(sv[i], s);
      widen(gv[i], g);
      load_weight<E>(a.w, c < D ? c : 0, w);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        ss = fmaf(s[j], s[j], ss);
        inner = fmaf(g[j] * w[j], s[j], inner);
      }
    }
    const float r = rsqrtf(row_sum<W>(ss, part, k) * a.inv_width + a.eps);
    const float m = row_sum<W>(inner, part, k + 1) * a.inv_width * r;    // mean(w dy v)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * W * 64 + lane) * E;
      float s[E], g[E], h[E], w[E];
      widen(sv[i], s);
      widen(gv[i], g);
      widen(hv[i], h);
      load_weight<E>(a.w, c < D ? c : 0, w);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float v = s[j] * r;
        dw[i][j] = fmaf(g[j], v, dw[i][j]);
        h[j] = fmaf(r, g[j] * w[j] - v * m, h[j]);
      }
      if (c < D) store16(static_cast<T *>(a.y) + base + c, narrow(h));
    }
  }
  if (!a.part) return;
  if constexpr (W == 1) {      // over the workgroup's waves, in order
    __shared__ __align__(16) float sum[3][64][E];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * 64 + lane) * E;
      __syncthreads();
      if (wave) {
#pragma unroll
        for (int j = 0; j < E; ++j) sum[wave - 1][lane][j] = dw[i][j];
      }
      __syncthreads();
      if (wave == 0 && c < D) {
#pragma unroll
        for (int j = 0; j < E; ++j) dw[i][j] = ((dw[i][j] + sum[0][lane][j]) + sum[1][lane][j]) + sum[2][lane][j];
        store_f32<E>(a.part + (size_t)blockIdx.x * D + c, dw[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * W * 64 + lane) * E;
      if (c < D) store_f32<E>(a.part + (size_t)blockIdx.x * D + c, dw[i]);
    }
  }
}

constexpr int FWD_BLOCKS = 1 << 18;     // a launch holds less than 2^32 threads
constexpr int BWD_BLOCKS = 1024;        // four workgroups a compute unit, each with its sums for the weight

int blocks_of(int tokens, int rows, int most) {
  const int n = (int)(((int64_t)tokens + rows - 1) / rows);
  return n < most ? n : most;
}
// one wave holds up to 8 x 64 x 16 bytes of a row
bool one_wave(bool bf16, int width) { return width <= (bf16 ? 4096 : 2048); }

// Calls f<W, V> for rows of this width: V is the next power of two that holds them.
template <typename T, typename F> hipError_t by_width(int width, F f) {
  constexpr int E = PER16<T>;
  if (width <= 64 * E) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
  if (width <= 128 * E) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 2>());
  if (width <= 256 * E) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
  if (width <= 512 * E) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
  if (width <= 1024 * E) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
  if (width <= 2048 * E) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
  if (width <= 4096 * E) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 16>());
  return hipErrorInvalidValue;
}

template <typename T> hipError_t fwd(bool q8, const NormArgs &a, hipStream_t s) {
  return by_width<T>(a.width, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    const int grid = blocks_of(a.tokens, 4 / W, FWD_BLOCKS);
    if (q8) hipLaunchKernelGGL((norm_fwd<T, W, V, true>), dim3(grid), dim3(THR), 0, s, a);
    else hipLaunchKernelGGL((norm_fwd<T, W, V, false>), dim3(grid), dim3(THR), 0, s, a);
    return hipGetLastError();
  });
}

template <typename T> hipError_t bwd(const NormArgs &a, int blocks, hipStream_t s) {
  return by_width<T>(a.width, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    hipLaunchKernelGGL((norm_bwd<T, W, V>), dim3(blocks), dim3(THR), 0, s, a);
    return hipGetLastError();
  });
}

int bwd_blocks(bool bf16, int tokens, int width) {
  return blocks_of(tokens, one_wave(bf16, width) ? 4 : 1, BWD_BLOCKS);
}

}  // namespace

size_t norm_bwd_workspace(bool bf16, int tokens, int width) {
  return (size_t)bwd_blocks(bf16, tokens, width) * width * sizeof(float);
}

hipError_t launch_norm_fwd(bool bf16, bool q8, NormArgs a, hipStream_t s) {
  a.inv_width = 1.f / a.width;
  return bf16 ? fwd<__bf16>(q8, a, s) : fwd<float>(q8, a, s);
}

hipError_t launch_norm_bwd(bool bf16, NormArgs a, float *dw, void *ws, hipStream_t s) {
  a.inv_width = 1.f / a.width;
  a.part = dw ? static_cast<float *>(ws) : nullptr;
  const int blocks = bwd_blocks(bf16, a.tokens, a.width);
  const hipError_t e = bf16 ? bwd<__bf16>(a, blocks, s) : bwd<float>(a, blocks, s);
  if (e != hipSuccess || !dw) return e;
  return launch_column_sum(a.part, blocks, a.width, dw, a.width, nullptr, s);
}

}  // namespace falcon
