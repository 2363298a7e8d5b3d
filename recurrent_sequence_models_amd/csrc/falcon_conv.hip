// Short causal convolution over time, one filter a channel, on gfx950, forward, backward and for
// single tokens.
//
//   p_t = b + sum_{j < W} w_j x_{t-W+1+j},  y_t = p_t or silu(p_t) = p_t sigmoid(p_t)
// where the W - 1 inputs before a sequence's first token are its initial state, and its last W - 1
// inputs its final one.  Backward, with d_t = dy_t act'(p_t):
//   dx_t = sum_j w_j d_{t+W-1-j} (within the sequence),  dw_j = sum_t d_t x_{t-W+1+j},  db = sum_t d_t.
//
// A thread owns 16 bytes of channels and a run of consecutive tokens, and slides over them with the
// last W - 1 inputs (backward: and the W unfinished gradients) in registers.  The W - 1 tokens next to
// a run are read again, from the cache as a rule: the runs beside belong to the same workgroup.
// In the backward pass d is formed again for the W - 1 tokens behind the run, rather than
// exchanged.  Bound: HBM, x and y (backward: x, dy and dx) once.
#include "block_kernels.h"
#include "row_io.h"

namespace falcon {
namespace {

constexpr int THR = 256, LANES = 16, RUNS = THR / LANES;   // lanes side by side over channels; runs of a workgroup
constexpr int AHEAD = 4;                                   // tokens whose loads are in flight together

template <int E> __device__ __forceinline__ float conv_at(const float (&w)[E], const float (&x)[E], int j) { return w[j] * x[j]; }

// This thread's filters: w[k][j] of tap k, channel j; bias.
template <int W, int E>
__device__ __forceinline__ void load_filters(const ConvArgs &a, int c, float (&w)[W][E], float (&b)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][j] = a.w[(size_t)(c + j) * W + k];
    b[j] = a.bias ? a.bias[c + j] : 0.f;
  }
}

// The W - 1 inputs before token t of sequence n, which begins at s.
template <typename T, int W>
__device__ __forceinline__ void load_window(const ConvArgs &a, int n, int s, int t, int c, u4 (&win)[W - 1]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int p = t - (W - 1) + i;
    if (p >= s) win[i] = load16(static_cast<const T *>(a.x) + (int64_t)p * a.ldx + c);
    else if (a.init) win[i] = load16(static_cast<const T *>(a.init) + ((size_t)n * (W - 1) + (p - s + W - 1)) * a.D + c);
    else win[i] = u4{0, 0, 0, 0};
  }
}

// b + sum of the window and the newest input
template <int W, int E>
__device__ __forceinline__ void convolve(const float (&w)[W][E], const float (&b)[E], const u4 (&win)[W - 1], const u4 &x,
                                         float (&p)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) p[j] = b[j];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float v[E];
    widen(k < W - 1 ? win[k < W - 1 ? k : 0] : x, v);
#pragma unroll
    for (int j = 0; j < E; ++j) p[j] = fmaf(w[k][j], v[j], p[j]);
  }
}

template <int W> __device__ __forceinline__ void slide(u4 (&win)[W - 1], const u4 &x) {
#pragma unroll
  for (int i = 0; i + 1 < W - 1; ++i) win[i] = win[i + 1];
  win[W - 2] = x;
}

// Rows of an [n, W - 1, D] array that belong to empty sequences, copied (zeros without a source).
template <typename T, int W>
__device__ __forceinline__ void copy_empty(const ConvArgs &a, const void *from, void *to, int first, int step, int c) {
  if (!a.seq.cu || !to) return;
  for (int n = first; n < a.seq.n; n += step) {
    if (a.seq.begin(n) < a.seq.end(n)) continue;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const size_t at = ((size_t)n * (W - 1) + i) * a.D + c;
      store16(static_cast<T *>(to) + at, from ? load16(static_cast<const T *>(from) + at) : u4{0, 0, 0, 0});
    }
  }
}

template <typename T, int W> __global__ __launch_bounds__(THR) void conv_fwd(ConvArgs a) {
  constexpr int E = PER16<T>;
  const int c = (blockIdx.y * LANES + threadIdx.x % LANES) * E;
  const int run = blockIdx.x * RUNS + threadIdx.x / LANES, total = a.seq.tokens();
  if (c >= a.D) return;
  float w[W][E], b[E];
  load_filters<W, E>(a, c, w, b);
  copy_empty<T, W>(a, a.init, a.final_state, run, gridDim.x * RUNS, c);
  const int64_t t0 = (int64_t)run * a.run;
  if (t0 >= total) return;
  const int last = (int)min(t0 + a.run, (int64_t)total);
  int t = (int)t0;
  for (int n = a.seq.of(t); n < a.seq.n && t < last; ++n) {
    const int s = a.seq.begin(n), e = a.seq.end(n), to = min(e, last);
    t = max(t, s);
    if (t >= to) continue;
    u4 win[W - 1];
    load_window<T, W>(a, n, s, t, c, win);
    for (; t < to; t += AHEAD) {
      u4 x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) x[i] = load16(static_cast<const T *>(a.x) + (int64_t)min(t + i, to - 1) * a.ldx + c);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (t + i < to) {
          float p[E];
          convolve<W, E>(w, b, win, x[i], p);
          if (a.silu) {
#pragma unroll
            for (int j = 0; j < E; ++j) p[j] *= sigmoid(p[j]);
          }
          store16(static_cast<T *>(a.y) + (size_t)(t + i) * a.D + c, narrow(p));
          slide<W>(win, x[i]);
        }
      }
    }
    t = to;
    if (to == e && a.final_state) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
        store16(static_cast<T *>(a.final_state) + ((size_t)n * (W - 1) + i) * a.D + c, win[i]);
    }
  }
}

template <typename T, int W> __global__ __launch_bounds__(THR) void conv_bwd(ConvArgs a) {
  constexpr int E = PER16<T>;
  const int col = threadIdx.x % LANES, c = (blockIdx.y * LANES + col) * E;
  const int run = blockIdx.x * RUNS + threadIdx.x / LANES, total = a.seq.tokens();
  const bool in = c < a.D;
  float w[W][E], b[E], dw[W][E] = {}, db[E] = {};
  if (in) {
    load_filters<W, E>(a, c, w, b);
    copy_empty<T, W>(a, a.d_final, a.d_init, run, gridDim.x * RUNS, c);
  }
  const int64_t t0 = (int64_t)run * a.run;
  const int last = (int)min(t0 + a.run, (int64_t)total);
  int t = (int)min(t0, (int64_t)total);
  if (in && t < last) {
    for (int n = a.seq.of(t); n < a.seq.n && t < last; ++n) {
      const int s = a.seq.begin(n), e = a.seq.end(n), to = min(e, last);   // own tokens: t .. to - 1
      t = max(t, s);
      if (t >= to) continue;
      const int from = t, upto = (int)min((int64_t)to + W - 1, (int64_t)e);
      u4 win[W - 1];
      load_window<T, W>(a, n, s, t, c, win);
      float acc[W][E] = {};      // acc[i]: the gradient of token t - (W - 1) + i so far
      // token p is finished: its gradient leaves, for the initial state where p lies before the sequence
      auto emit = [&](int p, const float (&v)[E]) {
        if (p >= from && p < to) store16(static_cast<T *>(a.dx) + (int64_t)p * a.lddx + c, narrow(v));
        else if (p < s && from == s && a.d_init)
          store16(static_cast<T *>(a.d_init) + ((size_t)n * (W - 1) + (p - s + W - 1)) * a.D + c, narrow(v));
      };
      for (; t < upto; t += AHEAD) {
        u4 x[AHEAD], g[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int q = min(t + i, upto - 1);
          x[i] = load16(static_cast<const T *>(a.x) + (int64_t)q * a.ldx + c);
          g[i] = load16(static_cast<const T *>(a.dy) + (size_t)q * a.D + c);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (t + i < upto) {
            float d[E], v[E];
            widen(g[i], d);
            if (a.silu) {
              float p[E];
              convolve<W, E>(w, b, win, x[i], p);
#pragma unroll
              for (int j = 0; j < E; ++j) {
                const float sg = sigmoid(p[j]);
                d[j] *= sg * fmaf(p[j], 1.f - sg, 1.f);
              }
            }
            if (t + i < to) {
#pragma unroll
              for (int k = 0; k < W; ++k) {
                widen(k < W - 1 ? win[k < W - 1 ? k : 0] : x[i], v);
#pragma unroll
                for (int j = 0; j < E; ++j) dw[k][j] = fmaf(d[j], v[j], dw[k][j]);
              }
#pragma unroll
              for (int j = 0; j < E; ++j) db[j] += d[j];
            }
#pragma unroll
            for (int k = 0; k < W; ++k)
#pragma unroll
              for (int j = 0; j < E; ++j) acc[k][j] = fmaf(w[k][j], d[j], acc[k][j]);
            emit(t + i - (W - 1), acc[0]);
#pragma unroll
            for (int k = 0; k + 1 < W; ++k)
#pragma unroll
              for (int j = 0; j < E; ++j) acc[k][j] = acc[k + 1][j];
#pragma unroll
            for (int j = 0; j < E; ++j) acc[W - 1][j] = 0.f;
            slide<W>(win, x[i]);
          }
        }
      }
      if (upto == e) {           // the sequence's end: its last inputs are its final state
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          if (a.d_final) {
            float v[E];
            widen(load16(static_cast<const T *>(a.d_final) + ((size_t)n * (W - 1) + i) * a.D + c), v);
#pragma unroll
            for (int j = 0; j < E; ++j) acc[i][j] += v[j];
          }
          emit(e - (W - 1) + i, acc[i]);
        }
      }
      t = to;
    }
  }
  if (!a.part) return;
  // the workgroup's sums for the weights, over its runs in order
  __shared__ __align__(16) float sum[RUNS][LANES][E];
  float *out = a.part + (size_t)blockIdx.x * a.D * (W + 1);
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) sum[threadIdx.x / LANES][col][j] = k < W ? dw[k < W ? k : 0][j] : db[j];
    __syncthreads();
    const int cc = blockIdx.y * LANES * E + threadIdx.x;
    if (threadIdx.x < LANES * E && cc < a.D) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) v += sum[r][threadIdx.x / E][threadIdx.x % E];
      out[k < W ? (size_t)cc * W + k : (size_t)a.D * W + cc] = v;
    }
  }
}

template <typename T, int W> __global__ __launch_bounds__(THR) void conv_step(ConvArgs a) {
  constexpr int E = PER16<T>;
  const int per = a.D / E;
  const int64_t i = (int64_t)blockIdx.x * THR + threadIdx.x;
  const int n = (int)(i / per), c = (int)(i - (int64_t)n * per) * E;
  if (n >= a.seq.n) return;
  u4 win[W - 1];
  const u4 x = load16(static_cast<const T *>(a.x) + (int64_t)n * a.ldx + c);
  const size_t at = (size_t)n * (W - 1) * a.D + c;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) win[k] = load16(static_cast<const T *>(a.init) + at + (size_t)k * a.D);
  float w[W][E], b[E], p[E];
  load_filters<W, E>(a, c, w, b);
  convolve<W, E>(w, b, win, x, p);
  if (a.silu) {
#pragma unroll
    for (int j = 0; j < E; ++j) p[j] *= sigmoid(p[j]);
  }
  store16(static_cast<T *>(a.y) + (size_t)n * a.D + c, narrow(p));
  slide<W>(win, x);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) store16(static_cast<T *>(a.final_state) + at + (size_t)k * a.D, win[k]);
}

// Tokens of a run: long runs read fewer tokens twice, short ones make more workgroups.
int run_of(SeqMap seq, int D, int E) {
  const int64_t cols = (D + LANES * E - 1) / (LANES * E);
  for (int run : {16, 8})
    if (((int64_t)seq.tokens() + run * RUNS - 1) / (run * RUNS) * cols >= 512) return run;
  return 4;
}
dim3 grid_of(SeqMap seq, int D, int E) {
  const int64_t per = (int64_t)run_of(seq, D, E) * RUNS;
  return dim3((unsigned)((seq.tokens() + per - 1) / per), (unsigned)((D + LANES * E - 1) / (LANES * E)));
}
int entries(bool bf16) { return bf16 ? 8 : 4; }

}  // namespace

bool conv_fits(bool bf16, SeqMap seq, int D) {
  const dim3 g = grid_of(seq, D, entries(bf16));
  return g.y <= 65535 && grid_fits((int64_t)g.x * g.y, THR);
}

size_t conv_bwd_workspace(bool bf16, int taps, SeqMap seq, int D) {
  return (size_t)grid_of(seq, D, entries(bf16)).x * D * (taps + 1) * sizeof(float);
}

#define FALCON_CONV(KERNEL, GRID)                                                                             \
  if (taps == 4 && bf16) hipLaunchKernelGGL((KERNEL<__bf16, 4>), GRID, dim3(THR), 0, s, a);                   \
  else if (taps == 4) hipLaunchKernelGGL((KERNEL<float, 4>), GRID, dim3(THR), 0, s, a);                       \
  else if (taps == 3 && bf16) hipLaunchKernelGGL((KERNEL<__bf16, 3>), GRID, dim3(THR), 0, s, a);              \
  else if (taps == 3) hipLaunchKernelGGL((KERNEL<float, 3>), GRID, dim3(THR), 0, s, a);                       \
  else if (taps == 2 && bf16) hipLaunchKernelGGL((KERNEL<__bf16, 2>), GRID, dim3(THR), 0, s, a);              \
  else if (taps == 2) hipLaunchKernelGGL((KERNEL<float, 2>), GRID, dim3(THR), 0, s, a);                       \
  else return hipErrorInvalidValue;

hipError_t launch_conv_fwd(bool bf16, int taps, ConvArgs a, hipStream_t s) {
  a.run = run_of(a.seq, a.D, entries(bf16));
  const dim3 grid = grid_of(a.seq, a.D, entries(bf16));
  FALCON_CONV(conv_fwd, grid)
  return hipGetLastError();
}

hipError_t launch_conv_bwd(bool bf16, int taps, ConvArgs a, float *dw, float *db, void *ws, hipStream_t s) {
  a.run = run_of(a.seq, a.D, entries(bf16));
  a.part = dw || db ? static_cast<float *>(ws) : nullptr;
  const dim3 grid = grid_of(a.seq, a.D, entries(bf16));
  FALCON_CONV(conv_bwd, grid)
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  return launch_column_sum(a.part, grid.x, (int64_t)a.D * (taps + 1), dw, (int64_t)a.D * taps, db, s);
}

hipError_t launch_conv_step(bool bf16, int taps, ConvArgs a, hipStream_t s) {
  const int64_t threads = (int64_t)a.seq.n * (a.D / entries(bf16));
  const dim3 grid((unsigned)((threads + THR - 1) / THR));
  FALCON_CONV(conv_step, grid)
  return hipGetLastError();
}
#undef FALCON_CONV

}  // namespace falcon
