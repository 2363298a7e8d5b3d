// Short causal convolution over time, one filter a channel, on gfx950, forward, backward and for
// single tokens.
//
//   p_t = b + sum_{j < W} w_j x_{t-W+1+j},  y_t = p_t or silu(p_t) = p_t sigmoid(p_t)
// where the W - 1 inputs before a sequence's first token are its initial state, and its last W - 1
// inputs its final one.  Backward, with d_t = dy_t act'(p_t):
//   dx_t = sum_j w_j d_{t+W-1-j} (within the sequence),  dw_j = sum_t d_t x_{t-W+1+j},  db = sum_t d_t.
//
// A thread owns E neighbouring channels (16 bytes; backward 4 channels, whose sums for the weights would else
// take the registers of half of the waves) and a run of consecutive tokens, and slides over them with the
// last W - 1 inputs (backward: and the W unfinished gradients) in registers.  The W - 1 tokens next to
// a run are read again, from the cache as a rule: the runs beside belong to the same workgroup.
// In the backward pass d is formed again for the W - 1 tokens behind the run, rather than
// exchanged.  Blocks of tokens inside a run need no comparisons (backward 3 of 39 us).  Bound: HBM, x and
// y (backward: x, dy and dx) once, and backward the vector unit beside it.
// Measured, 4 x 4096 x 1536 bf16, 4 taps, silu: forward 24 us (101 MB at 4.2 TB/s), backward 33 us (151 MB at 4.6) and 5 us
// to add the weights' gradients; 64 tokens x 4096: 3.9 us.
#include <type_traits>

#include "block_kernels.h"
#include "row_io.h"

namespace falcon {
namespace {

constexpr int THR = CONV_THR;
constexpr int AHEAD = 4;                                   // tokens whose loads are in flight together, W - 1 at least

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
template <typename T, int W, int E>
__device__ __forceinline__ void load_window(const ConvArgs &a, int n, int s, int t, int c, Few<T, E> (&win)[W - 1]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int p = t - (W - 1) + i;
    if (p >= s) fetch(static_cast<const T *>(a.x) + (int64_t)p * a.ldx + c, win[i]);
    else if (a.init) fetch(static_cast<const T *>(a.init) + ((size_t)n * (W - 1) + (p - s + W - 1)) * a.D + c, win[i]);
    else win[i] = Few<T, E>{};
  }
}

// b + sum of the window and the newest input
template <typename T, int W, int E>
__device__ __forceinline__ void convolve(const float (&w)[W][E], const float (&b)[E], const Few<T, E> (&win)[W - 1],
                                         const Few<T, E> &x, float (&p)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) p[j] = b[j];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const Few<T, E> v = k < W - 1 ? win[k < W - 1 ? k : 0] : x;
#pragma unroll
    for (int j = 0; j < E; ++j) p[j] = fmaf(w[k][j], v[j], p[j]);
  }
}

template <typename T, int W, int E> __device__ __forceinline__ void slide(Few<T, E> (&win)[W - 1], const Few<T, E> &x) {
#pragma unroll
  for (int i = 0; i + 1 < W - 1; ++i) win[i] = win[i + 1];
  win[W - 2] = x;
}

// Rows of an [n, W - 1, D] array that belong to empty sequences, copied (zeros without a source).
template <typename T, int W, int E>
__device__ __forceinline__ void copy_empty(const ConvArgs &a, const void *from, void *to, int first, int step, int c) {
  if (!a.seq.cu || !to) return;
  for (int n = first; n < a.seq.n; n += step) {
    if (a.seq.begin(n) < a.seq.end(n)) continue;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const size_t at = ((size_t)n * (W - 1) + i) * a.D + c;
      Few<T, E> v{};
      if (from) fetch(static_cast<const T *>(from) + at, v);
      put(static_cast<T *>(to) + at, v);
    }
  }
}

// The number of a thread's run, of LANES lanes each.
template <int LANES> __device__ __forceinline__ int run_of() {
  const int r = threadIdx.x / LANES;
  return blockIdx.x * (THR / LANES) + (LANES == 64 ? __builtin_amdgcn_readfirstlane(r) : r);
}

template <typename T, int W, int LANES> __global__ __launch_bounds__(THR) void conv_fwd(ConvArgs a) {
  constexpr int E = PER16<T>, RUNS = THR / LANES;
  const int c = (blockIdx.y * LANES + threadIdx.x % LANES) * E;
  const int run = run_of<LANES>(), total = a.seq.tokens();
  if (c >= a.D) return;
  float w[W][E], b[E];
  load_filters<W, E>(a, c, w, b);
  copy_empty<T, W, E>(a, a.init, a.final_state, run, gridDim.x * RUNS, c);
  const int64_t t0 = (int64_t)run * a.run;
  if (t0 >= total) return;
  const int last = (int)min(t0 + a.run, (int64_t)total);
  int t = (int)t0;
  for (int n = a.seq.of(t); n < a.seq.n && t < last; ++n) {
    const int s = a.seq.begin(n), e = a.seq.end(n), to = min(e, last);
    t = max(t, s);
    if (t >= to) continue;
    Few<T, E> win[W - 1];
    load_window<T, W, E>(a, n, s, t, c, win);
    // AHEAD tokens from t on; all of them exist, or (ends) those behind the last are left out
    auto block = [&](auto ends) __attribute__((always_inline)) {
      const T *from = static_cast<const T *>(a.x) + (int64_t)t * a.ldx + c;
      T *out = static_cast<T *>(a.y) + (size_t)t * a.D + c;
      Few<T, E> x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) fetch(from + (decltype(ends)::value ? min(i, to - 1 - t) : i) * a.ldx, x[i]);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (decltype(ends)::value && t + i >= to) continue;
        float p[E];
        convolve<T, W, E>(w, b, win, x[i], p);
        if (a.silu) {
#pragma unroll
          for (int j = 0; j < E; ++j) p[j] *= sigmoid(p[j]);
        }
        put(out + (size_t)i * a.D, p);
        slide<T, W, E>(win, x[i]);
      }
    };
    for (; t + AHEAD <= to; t += AHEAD) block(std::false_type());
    if (t < to) block(std::true_type());
    t = to;
    if (to == e && a.final_state) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
        put(static_cast<T *>(a.final_state) + ((size_t)n * (W - 1) + i) * a.D + c, win[i]);
    }
  }
}

template <typename T, int W> __global__ __launch_bounds__(THR) void conv_bwd(ConvArgs a) {
  constexpr int E = 4, LANES = CONV_WIDE, RUNS = THR / LANES;
  const int col = threadIdx.x % LANES, c = (blockIdx.y * LANES + col) * E;
  const int run = run_of<LANES>(), total = a.seq.tokens();
  const bool in = c < a.D;
  float w[W][E], b[E], dw[W][E] = {}, db[E] = {};
  if (in) {
    load_filters<W, E>(a, c, w, b);
    copy_empty<T, W, E>(a, a.d_final, a.d_init, run, gridDim.x * RUNS, c);
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
      Few<T, E> win[W - 1];
      load_window<T, W, E>(a, n, s, t, c, win);
      float acc[W][E] = {};      // acc[i]: the gradient of token t - (W - 1) + i so far
      // token p is finished: its gradient leaves, for the initial state where p lies before the sequence
      auto emit = [&](int p, const float (&v)[E]) {
        if (p >= from && p < to) put(static_cast<T *>(a.dx) + (int64_t)p * a.lddx + c, v);
        else if (p < s && from == s && a.d_init)
          put(static_cast<T *>(a.d_init) + ((size_t)n * (W - 1) + (p - s + W - 1)) * a.D + c, v);
      };
      // AHEAD tokens from t on; (ends) some may be behind the last, behind this thread's own, or finish one before those
      auto block = [&](auto ends) __attribute__((always_inline)) {
        constexpr bool ENDS = decltype(ends)::value;
        const T *px = static_cast<const T *>(a.x) + (int64_t)t * a.ldx + c;
        const T *pg = static_cast<const T *>(a.dy) + (size_t)t * a.D + c;
        T *out = static_cast<T *>(a.dx) + (int64_t)(t - (W - 1)) * a.lddx + c;
        Few<T, E> x[AHEAD], g[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int64_t q = ENDS ? min(i, upto - 1 - t) : i;
          fetch(px + q * a.ldx, x[i]);
          fetch(pg + q * a.D, g[i]);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (ENDS && t + i >= upto) continue;
          float d[E];
#pragma unroll
          for (int j = 0; j < E; ++j) d[j] = g[i][j];
          if (a.silu) {
            float p[E];
            convolve<T, W, E>(w, b, win, x[i], p);
#pragma unroll
            for (int j = 0; j < E; ++j) {
              const float sg = sigmoid(p[j]);
              d[j] *= sg * fmaf(p[j], 1.f - sg, 1.f);
            }
          }
          if (!ENDS || t + i < to) {
#pragma unroll
            for (int k = 0; k < W; ++k) {
              const Few<T, E> v = k < W - 1 ? win[k < W - 1 ? k : 0] : x[i];
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
          if constexpr (ENDS) emit(t + i - (W - 1), acc[0]);
          else put(out + i * a.lddx, acc[0]);
#pragma unroll
          for (int k = 0; k + 1 < W; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) acc[k][j] = acc[k + 1][j];
#pragma unroll
          for (int j = 0; j < E; ++j) acc[W - 1][j] = 0.f;
          slide<T, W, E>(win, x[i]);
        }
      };
      block(std::true_type());
      for (t += AHEAD; t + AHEAD <= to; t += AHEAD) block(std::false_type());
      for (; t < upto; t += AHEAD) block(std::true_type());
      if (upto == e) {           // the sequence's end: its last inputs are its final state
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          if (a.d_final) {
            Few<T, E> v;
            fetch(static_cast<const T *>(a.d_final) + ((size_t)n * (W - 1) + i) * a.D + c, v);
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

// Workgroups of one wave (64 x 4096 make 512, of 256 threads 128: fewer than compute units); those of a sequence follow
// each other.
constexpr int STEP_THR = 64;
__host__ __device__ inline int step_blocks(int D, int E) { return (D / E + STEP_THR - 1) / STEP_THR; }
template <typename T, int W> __global__ __launch_bounds__(STEP_THR) void conv_step(ConvArgs a) {
  constexpr int E = PER16<T>;
  const int per = step_blocks(a.D, E), n = blockIdx.x / per, c = ((blockIdx.x - n * per) * STEP_THR + threadIdx.x) * E;
  if (c >= a.D) return;
  Few<T, E> win[W - 1];
  Few<T, E> x;
  fetch(static_cast<const T *>(a.x) + (int64_t)n * a.ldx + c, x);
  const size_t at = (size_t)n * (W - 1) * a.D + c;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) fetch(static_cast<const T *>(a.init) + at + (size_t)k * a.D, win[k]);
  float w[W][E], b[E], p[E];
  load_filters<W, E>(a, c, w, b);
  convolve<T, W, E>(w, b, win, x, p);
  if (a.silu) {
#pragma unroll
    for (int j = 0; j < E; ++j) p[j] *= sigmoid(p[j]);
  }
  put(static_cast<T *>(a.y) + (size_t)n * a.D + c, p);
  slide<T, W, E>(win, x);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) put(static_cast<T *>(a.final_state) + at + (size_t)k * a.D, win[k]);
}

dim3 grid_of(const ConvPlan &p) { return dim3((unsigned)p.blocks, (unsigned)p.wide); }

template <typename T, int W> void fwd(const ConvPlan &p, const ConvArgs &a, hipStream_t s) {
  if (p.lanes == CONV_NARROW) hipLaunchKernelGGL((conv_fwd<T, W, CONV_NARROW>), grid_of(p), dim3(THR), 0, s, a);
  else hipLaunchKernelGGL((conv_fwd<T, W, CONV_WIDE>), grid_of(p), dim3(THR), 0, s, a);
}
template <typename T, int W> void bwd(const ConvPlan &p, const ConvArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((conv_bwd<T, W>), grid_of(p), dim3(THR), 0, s, a);
}
template <typename T, int W> void step(const ConvPlan &p, const ConvArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((conv_step<T, W>), grid_of(p), dim3(STEP_THR), 0, s, a);
}

}  // namespace

bool conv_step_fits(bool bf16, int n, int D) { return grid_fits((int64_t)n * step_blocks(D, bf16 ? 8 : 4), STEP_THR); }

bool conv_fits(bool bf16, SeqMap seq, int D) {
  for (const bool back : {false, true}) {
    const ConvPlan p = conv_plan(seq, D, bf16, back);
    if (p.wide > 65535 || !grid_fits(p.blocks * p.wide, THR)) return false;
  }
  return true;
}

size_t conv_bwd_workspace(bool bf16, int taps, SeqMap seq, int D) {
  return (size_t)conv_plan(seq, D, bf16, true).blocks * D * (taps + 1) * sizeof(float);
}

#define FALCON_CONV(PASS)                              \
  if (taps == 4 && bf16) PASS<__bf16, 4>(p, a, s);     \
  else if (taps == 4) PASS<float, 4>(p, a, s);         \
  else if (taps == 3 && bf16) PASS<__bf16, 3>(p, a, s); \
  else if (taps == 3) PASS<float, 3>(p, a, s);         \
  else if (taps == 2 && bf16) PASS<__bf16, 2>(p, a, s); \
  else if (taps == 2) PASS<float, 2>(p, a, s);         \
  else return hipErrorInvalidValue;

hipError_t launch_conv_fwd(bool bf16, int taps, ConvArgs a, hipStream_t s) {
  const ConvPlan p = conv_plan(a.seq, a.D, bf16, false);
  a.run = p.run;
  FALCON_CONV(fwd)
  return hipGetLastError();
}

hipError_t launch_conv_bwd(bool bf16, int taps, ConvArgs a, float *dw, float *db, void *ws, hipStream_t s) {
  const ConvPlan p = conv_plan(a.seq, a.D, bf16, true);
  a.run = p.run;
  a.part = dw || db ? static_cast<float *>(ws) : nullptr;
  FALCON_CONV(bwd)
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  return launch_column_sum(a.part, (int)p.blocks, (int64_t)a.D * (taps + 1), dw, (int64_t)a.D * taps, db, s);
}

hipError_t launch_conv_step(bool bf16, int taps, ConvArgs a, hipStream_t s) {
  const ConvPlan p = {STEP_THR, 1, (int64_t)a.seq.n * step_blocks(a.D, bf16 ? 8 : 4), 1};
  FALCON_CONV(step)
  return hipGetLastError();
}
#undef FALCON_CONV

}  // namespace falcon
