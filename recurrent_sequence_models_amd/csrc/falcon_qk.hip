// Query / key head norm with rotary positions on gfx950, forward and backward.
//
// A row is one head of one token, x in R^d.  With r = (mean x^2 + eps)^(-1/2):
//   z = x r w                               (norm; z = x without it)
//   pairs (z_a, z_b) of the first `rot` entries turn by the angle pos * freq_j:
//   y_a = s (z_a cos - z_b sin),  y_b = s (z_b cos + z_a sin)
//   (half layout: a = j, b = j + rot/2; interleaved: a = 2j, b = 2j + 1)
// and the rest passes.  The backward pass turns dy back, u = R^T dy, and then
//   dw = sum over rows of u x r,   dx = r w u - x r^3 mean(w u x).
//
// Bound: HBM, each row read once and written once.  A row is 16 bytes a lane, so its
// sums run over 4 to 32 neighbouring lanes.  The angles depend on the token and j alone:
// a workgroup computes the (cos, sin) of its tokens once into LDS and all their heads
// read them there (per row they would cost more instructions than everything else).
// pos * freq is reduced to a fraction of a turn in 64 bits: at position 10^6 a 32-bit
// product would be off by 2^-5 radians.
// Measured, where a plain copy moves 5.1 TB/s: forward, 16384 tokens, 12 + 12 heads of 64, bf16:
// 18.8 us (101 MB at 5.4 TB/s); backward, 16387 tokens, 16 + 4 heads of 128, bf16 with fp32
// incoming gradients: 68 us (336 MB at 4.9 TB/s) and 4.7 us to add the weights' gradients.
#include "layer_kernels.h"
#include "lane_ops.h"
#include "mfma_frag.h"

namespace falcon {
namespace {

constexpr int THR = 256;
// workgroups of the forward pass, at most (a launch holds less than 2^32 threads), and
constexpr int FWD_BLOCKS = 1 << 18;
// of the backward pass: four a compute unit, each with its sum for the weights (16387 tokens, 16 + 4
// heads of 128: 73 us; 768 workgroups 86, 2048 77)
constexpr int BWD_BLOCKS = 1024;

template <typename T> constexpr int EPL = 16 / (int)sizeof(T);   // entries per lane

__device__ __forceinline__ void load_row(const __bf16 *p, float (&o)[8]) {
  const bf8 v = *reinterpret_cast<const bf8 *>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (float)v[j];
}
template <int N> __device__ __forceinline__ void load_row(const float *p, float (&o)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const f4 v = *reinterpret_cast<const f4 *>(p + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j + i] = v[i];
  }
}
// bf16 results are rounded once, to nearest even.
__device__ __forceinline__ void store_row(__bf16 *p, const float (&v)[8]) {
  bf8 b;
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = (__bf16)v[j];
  *reinterpret_cast<bf8 *>(p) = b;
}
__device__ __forceinline__ void store_row(float *p, const float (&v)[4]) {
  *reinterpret_cast<f4 *>(p) = f4{v[0], v[1], v[2], v[3]};
}

// Sum over the L lanes of a row, in each of them.
template <int L> __device__ __forceinline__ float row_sum(float x) {
  x = lane_sum<(L < 16 ? L : 16)>(x);
  if constexpr (L == 32) x = add_xor16(x);
  return x;
}

// (cos, sin) times the scale for `n` tokens from t0 into tab[token][j].
__device__ __forceinline__ void fill_table(const QkArgs &a, int t0, int n, float2 *tab) {
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < n * half; i += THR) {
    const int t = i / half, j = i - t * half;
    const double turns = (double)a.pos[t0 + t] * a.freq[j] * 0.15915494309189533577;   // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    tab[i] = float2{c * a.scale, s * a.scale};
  }
}

// Where a lane's entries stand in the rotation, the same for every row: the lane that
// holds its partners (half layout), and its first angle.
struct Turn { int lane, j0; bool on, upper; };

template <typename T, int D> __device__ __forceinline__ Turn turn_of(const QkArgs &a) {
  constexpr int E = EPL<T>, L = D / E;
  const int lane = threadIdx.x & 63, e0 = (lane % L) * E, half = a.rot / 2;
  Turn t;
  t.on = e0 < a.rot;
  t.upper = !a.interleaved && e0 >= half;
  t.j0 = a.interleaved ? e0 / 2 : (t.upper ? e0 - half : e0);
  t.lane = lane;
  if (!a.interleaved && t.on) t.lane = t.upper ? lane - half / E : lane + half / E;
  return t;
}

// z <- R z (BACK: R^T z) for this lane's entries; every lane of the wave calls it.
template <bool BACK, int E>
__device__ __forceinline__ void rotate(float (&z)[E], const Turn &t, const float2 *tab, bool interleaved) {
  if (interleaved) {
    if (!t.on) return;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 cs = tab[t.j0 + i];
      const float s = BACK ? -cs.y : cs.y, p = z[2 * i], q = z[2 * i + 1];
      z[2 * i] = p * cs.x - q * s;
      z[2 * i + 1] = q * cs.x + p * s;
    }
    return;
  }
  float o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = __shfl(z[i], t.lane);
  if (!t.on) return;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float2 cs = tab[t.j0 + i];
    const float s = t.upper != BACK ? cs.y : -cs.y;
    z[i] = z[i] * cs.x + o[i] * s;
  }
}

template <int E> __device__ __forceinline__ void load_weight(const float *w, int e0, float (&o)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) o[j] = 1.f;
  if (w) load_row<E>(w + e0, o);
}

template <typename T, int D> __global__ __launch_bounds__(THR) void qk_fwd(QkArgs a) {
  constexpr int E = EPL<T>, L = D / E, ROWS = THR / L;
  extern __shared__ __align__(16) float2 tab[];
  const int H = a.hq + a.hk, e0 = (threadIdx.x % L) * E;
  const Turn turn = turn_of<T, D>(a);
  float w[2][E];
  load_weight<E>(a.w[0], e0, w[0]);
  load_weight<E>(a.w[1], e0, w[1]);
  for (int t0 = blockIdx.x * a.tok; t0 < a.tokens; t0 += gridDim.x * a.tok) {
    const int nt = min(a.tok, a.tokens - t0), rows = nt * H;
    if (t0 >= (int)gridDim.x * a.tok) __syncthreads();   // the table of the tokens before is read no more
    fill_table(a, t0, nt, tab);
    __syncthreads();
    for (int base = 0; base < rows; base += ROWS) {   // the same count for every wave: rotate() needs whole waves
      const int row = base + threadIdx.x / L;
      const bool on = row < rows;
      const int t = on ? row / H : 0, hh = on ? row - t * H : 0;
      const bool isk = hh >= a.hq;
      const int64_t head = (int64_t)(isk ? hh - a.hq : hh) * D + e0;
      const QkTensor &xs = a.x[isk], &ys = a.y[isk];
      float z[E];
      load_row(static_cast<const T *>(xs.p) + (t0 + t) * xs.ld + head, z);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(z[j], z[j], ss);
        const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < E; ++j) z[j] *= r * (isk ? w[1][j] : w[0][j]);
      }
      rotate<false, E>(z, turn, tab + t * (a.rot / 2), a.interleaved);
      if (on) store_row(static_cast<T *>(const_cast<void *>(ys.p)) + (t0 + t) * ys.ld + head, z);
    }
  }
}

// T: inputs and their gradients; G: incoming gradients.
template <typename T, typename G, int D> __global__ __launch_bounds__(THR) void qk_bwd(QkArgs a) {
  constexpr int E = EPL<T>, L = D / E, ROWS = THR / L;
  extern __shared__ __align__(16) float2 tab[];
  const int H = a.hq + a.hk, e0 = (threadIdx.x % L) * E;
  const Turn turn = turn_of<T, D>(a);
  float w[2][E], dw[2][E] = {};
  load_weight<E>(a.w[0], e0, w[0]);
  load_weight<E>(a.w[1], e0, w[1]);
  for (int t0 = blockIdx.x * a.tok; t0 < a.tokens; t0 += gridDim.x * a.tok) {
    const int nt = min(a.tok, a.tokens - t0), rows = nt * H;
    __syncthreads();                     // the table of the tokens before is read no more
    fill_table(a, t0, nt, tab);
    __syncthreads();
    for (int base = 0; base < rows; base += ROWS) {
      const int row = base + threadIdx.x / L;
      const bool on = row < rows;
      const int t = on ? row / H : 0, hh = on ? row - t * H : 0;
      const bool isk = hh >= a.hq;
      const int64_t head = (int64_t)(isk ? hh - a.hq : hh) * D + e0;
      const QkTensor &xs = a.x[isk], &gs = a.dy[isk], &ys = a.y[isk];
      float u[E];
      load_row(static_cast<const G *>(gs.p) + (t0 + t) * gs.ld + head, u);
      rotate<true, E>(u, turn, tab + t * (a.rot / 2), a.interleaved);
      if (a.norm) {
        float x[E], ss = 0.f, inner = 0.f;
        load_row(static_cast<const T *>(xs.p) + (t0 + t) * xs.ld + head, x);
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
        const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float xr = x[j] * r, g = on ? u[j] * xr : 0.f;
          dw[0][j] += isk ? 0.f : g;
          dw[1][j] += isk ? g : 0.f;
          u[j] *= isk ? w[1][j] : w[0][j];
          x[j] = xr;
          inner = fmaf(u[j], xr, inner);
        }
        const float m = row_sum<L>(inner) * (1.f / D);
#pragma unroll
        for (int j = 0; j < E; ++j) u[j] = r * (u[j] - x[j] * m);
      }
      if (on) store_row(static_cast<T *>(const_cast<void *>(ys.p)) + (t0 + t) * ys.ld + head, u);
    }
  }
  if (!a.part) return;
  // the workgroup's weight gradients: over its ROWS row groups, in order
  __shared__ float sum[ROWS][D];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) sum[threadIdx.x / L][e0 + j] = dw[k][j];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll 8
      for (int i = 0; i < ROWS; ++i) s += sum[i][threadIdx.x];
      a.part[((size_t)blockIdx.x * 2 + k) * D + threadIdx.x] = s;
    }
  }
}

// Sums the workgroups' weight gradients, in a fixed order: block (16 entries, tensor), 64
// slices of the workgroups for each entry.
constexpr int SUM_E = 16, SUM_S = 1024 / SUM_E;
__global__ __launch_bounds__(1024) void qk_weight_sum(QkArgs a, int d, int blocks) {
  __shared__ float sum[SUM_S][SUM_E];
  const int k = blockIdx.y, e = threadIdx.x % SUM_E, sl = threadIdx.x / SUM_E, col = blockIdx.x * SUM_E + e;
  float s = 0.f;
#pragma unroll 4
  for (int i = sl; i < blocks; i += SUM_S) s += a.part[((size_t)i * 2 + k) * d + col];
  sum[sl][e] = s;
  __syncthreads();
  if (threadIdx.x < SUM_E && a.dw[k]) {
    s = 0.f;
#pragma unroll 8
    for (int i = 0; i < SUM_S; ++i) s += sum[i][e];
    a.dw[k][col] = s;
  }
}

int blocks_of(int tokens, int tok, int most) {
  const int n = (tokens + tok - 1) / tok;
  return n < most ? n : most;
}

// Tokens of a workgroup: they share the table's work and the barrier, and fewer tokens leave
// more workgroups.  1 / 2 / 4 tokens a workgroup took, forward, 12 + 12 heads of 64, bf16:
//   512 and fewer do not fill the chip: 64 tokens 2.8 / 3.4 / 4.1 us
//   1024 tokens 3.9 / 4.1 / 4.6 us (16 + 4 heads of 128: 6.1 / 5.4 / 6.4; backward 12.2 / 10.2 / 11.1)
//   2048 tokens 5.6 / 5.7 / 5.7 us (16 + 4 heads of 128: 9.9 / 8.7 / 8.5; fp32, 12 + 12 of 64: 7.2 / 6.9 / 8.2)
//   4096 tokens 9.3 / 8.7 / 7.8 us (16 + 4 heads of 128: 15.2 / 13.2 / 11.8), 32768 tokens 60 / 48 / 39 us
int tokens_per_block(int tokens) { return tokens >= 4096 ? 4 : tokens >= 1024 ? 2 : 1; }

}  // namespace

size_t qk_bwd_workspace(int tokens, int d) {
  return (size_t)blocks_of(tokens, tokens_per_block(tokens), BWD_BLOCKS) * 2 * d * sizeof(float);
}

hipError_t launch_qk_fwd(bool bf16, int d, QkArgs a, hipStream_t s) {
  a.tok = tokens_per_block(a.tokens);
  const int grid = blocks_of(a.tokens, a.tok, FWD_BLOCKS);
  const unsigned lds = a.tok * (a.rot / 2) * sizeof(float2);
#define FALCON_QK(D_)                                                                                        \
  if (d == D_) {                                                                                             \
    if (bf16) hipLaunchKernelGGL((qk_fwd<__bf16, D_>), dim3(grid), dim3(THR), lds, s, a);                    \
    else hipLaunchKernelGGL((qk_fwd<float, D_>), dim3(grid), dim3(THR), lds, s, a);                          \
    return hipGetLastError();                                                                                \
  }
  FALCON_QK(32)
  FALCON_QK(64)
  FALCON_QK(128)
#undef FALCON_QK
  return hipErrorInvalidValue;
}

hipError_t launch_qk_bwd(bool bf16, bool dy_f32, int d, QkArgs a, void *ws, hipStream_t s) {
  a.tok = tokens_per_block(a.tokens);
  const bool weights = a.norm && (a.dw[0] || a.dw[1]);
  a.part = weights ? static_cast<float *>(ws) : nullptr;
  const int blocks = blocks_of(a.tokens, a.tok, BWD_BLOCKS);
  const unsigned lds = a.tok * (a.rot / 2) * sizeof(float2);
#define FALCON_QK(D_)                                                                                            \
  if (d == D_) {                                                                                                 \
    if (!bf16) hipLaunchKernelGGL((qk_bwd<float, float, D_>), dim3(blocks), dim3(THR), lds, s, a);               \
    else if (dy_f32) hipLaunchKernelGGL((qk_bwd<__bf16, float, D_>), dim3(blocks), dim3(THR), lds, s, a);        \
    else hipLaunchKernelGGL((qk_bwd<__bf16, __bf16, D_>), dim3(blocks), dim3(THR), lds, s, a);                   \
    const hipError_t e = hipGetLastError();                                                                      \
    if (e != hipSuccess || !weights) return e;                                                                   \
    hipLaunchKernelGGL(qk_weight_sum, dim3(D_ / SUM_E, 2), dim3(1024), 0, s, a, D_, blocks);                     \
    return hipGetLastError();                                                                                    \
  }
  FALCON_QK(32)
  FALCON_QK(64)
  FALCON_QK(128)
#undef FALCON_QK
  return hipErrorInvalidValue;
}

}  // namespace falcon
