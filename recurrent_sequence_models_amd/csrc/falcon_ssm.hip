// Selective state-space scan on gfx950, forward and for single tokens.
//
// Per sequence, channel d and state n, with delta_t = softplus(dt_t + bias) (or dt_t + bias):
//   h_t = exp(delta_t A_dn) h_{t-1} + delta_t x_t B_tn
//   y_t = (sum_n C_tn h_t + D_d x_t) silu(z_t)
//
// A tile's steps pass through LDS once: (delta, delta x) of its channels, B and C.  The waves of a
// workgroup that lie behind each other in time each compose their 16 steps first, h -> P h + H
// with P = exp(A sum of delta), keeping the 64 decays of a lane in registers; then every wave
// joins the maps before its own to the tile's first state and runs its steps again from there,
// without an exponential.  So time gives 4 times the waves that the channels alone would, for 7
// instructions a state and step (one of them the exponential) where a plain recurrence pays 5.
//
// Few long sequences: they are cut into segments, whose maps a pass of its own forms, and which then
// run in parallel.
//
// Bound: the vector unit: 44 instructions (49 issue slots) for 4 states and a step, with what a tile's loading, softplus,
// gate and joins cost; busy 91 % of the time.  Measured, bf16: 8 x 2048 x 1536, N = 16: 146 us among other work (2.8e12
// states a second; the bytes alone would take 43 us), 160 in a row, where the card's clock is lower; 8 x 2048 x 768, N = 32:
// 217, 64: 347; single tokens, 64 x 4096: 9 us (36 MB at 4.0 TB/s).
#include "ssm_common.h"

namespace falcon {
namespace {

// MAPS: only the segment's map (end state from zero, sum of delta) is formed.
template <typename T, int N, int TW, int STEPS, bool MAPS>
__global__ __launch_bounds__((SsmTile<N, SSM_FWD_CH, TW, STEPS>::THR), (STEPS == 16 ? 3 : 4)) void ssm_fwd(SsmArgs a) {
  typedef SsmTile<N, SSM_FWD_CH, TW, STEPS> L;
  constexpr int V = L::VEC, BV = L::BV, CH = SSM_FWD_CH;
  __shared__ __align__(16) float2 step[L::TS][CH];        // (delta, delta x); then (y, -)
  __shared__ __align__(16) float sB[L::TS][N], sC[L::TS][N];
  __shared__ __align__(16) float mapP[TW][CH][N], mapH[TW][CH][N];
  __shared__ float sumd[TW][CH];
  const int groups = (a.D + CH - 1) / CH;
  const SsmPlace place = ssm_place(groups, slots_of(a.seq, a.seg));
  if (!place.any) return;
  const Segment g = find_segment(a.seq, a.seg, place.slot);
  const int c0 = place.group * CH;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tw = wave / L::WIDE, ch = (wave % L::WIDE) * L::CW + lane / L::P, p4 = (lane % L::P) * 4;
  const int c = c0 + ch;                      // this lane's channel
  const bool on = c < a.D;
  // an empty sequence has one slot, in which it ends where it began
  if (!g.any && !(g.s == g.e && g.slot == first_slot(a.seq, g.n, a.seg))) return;
  const bool first = g.t0 == g.s, lastseg = g.t1 == g.e;
  if constexpr (MAPS) { if (lastseg) return; }      // nobody starts from its end
  f4 A2{0.f, 0.f, 0.f, 0.f}, h{0.f, 0.f, 0.f, 0.f};
  if (on) {
    A2 = *reinterpret_cast<const f4 *>(a.A + (size_t)c * N + p4) * SSM_LOG2E;
    if constexpr (!MAPS) {
      if (!first) h = *reinterpret_cast<const f4 *>(a.seg_state + ((size_t)g.slot * a.D + c) * N + p4);
      else if (a.init) h = *reinterpret_cast<const f4 *>(a.init + ((size_t)g.n * a.D + c) * N + p4);
    }
  }
  // the part of a tile that this thread loads, and of y that it stores
  const int ls = tid / (CH / V), lc = (tid % (CH / V)) * V, lcc = c0 + lc;
  const bool lon = lcc < a.D;
  const int bs = tid / (N / BV), bn = (tid % (N / BV)) * BV;
  float bias[V] = {}, skip[V] = {};
  if (lon) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (a.bias) bias[j] = a.bias[lcc + j];
      if (a.skip) skip[j] = a.skip[lcc + j];
    }
  }
  const int chunk0 = MAPS ? 0 : first_slot(a.seq, g.n, SSM_CHUNK<N>);
  Few<T, V> nx, nd, nz;                       // the next tile's entries of this thread
  Few<T, BV> nB, nC;
  auto load = [&](int t) {
    const int q = min(ls, g.t1 - 1 - t), qb = min(bs, g.t1 - 1 - t), cc = lon ? lcc : 0;
    fetch(entry<T>(a.x, a.ldx, t, q, cc), nx);
    fetch(entry<T>(a.dt, a.lddt, t, q, cc), nd);
    if (!MAPS && a.z) fetch(entry<T>(a.z, a.ldz, t, q, cc), nz);
    fetch(entry<T>(a.B, a.ldB, t, qb, bn), nB);
    if (!MAPS) fetch(entry<T>(a.C, a.ldC, t, qb, bn), nC);
  };
  float total = 0.f;                          // MAPS: the sum of delta of this lane's channel
  if (g.any) load(g.t0);
  for (int t = g.t0; t < g.t1; t += L::TS) {
    const Few<T, V> x = nx, z = nz;
    const bool valid = lon && t + ls < g.t1;      // steps behind the end change nothing: delta = 0
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d = nd[j] + bias[j];
      if (a.softplus) d = softplus(d);
      step[ls][lc + j] = valid ? float2{d, d * x[j]} : float2{0.f, 0.f};
    }
    const bool there = t + bs < g.t1;             // and B = 0: the last token's may be infinite
#pragma unroll
    for (int j = 0; j < BV; ++j) {
      sB[bs][bn + j] = there ? nB[j] : 0.f;
      if constexpr (!MAPS) sC[bs][bn + j] = nC[j];
    }
    __syncthreads();
    if (t + L::TS < g.t1) load(t + L::TS);
    const int s0 = tw * STEPS;
    f4 dec[STEPS];
    f4 run = h;                                // the state before this wave's steps
    if constexpr (TW > 1 || MAPS) {
      f4 H{0.f, 0.f, 0.f, 0.f}, Pm;
      float sd = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const float2 du = step[s0 + s][ch];
        const f4 b = *reinterpret_cast<const f4 *>(&sB[s0 + s][p4]);
        sd += du.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dec[s][j] = __builtin_amdgcn_exp2f(du.x * A2[j]);
          H[j] = fmaf(dec[s][j], H[j], du.y * b[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) Pm[j] = __builtin_amdgcn_exp2f(sd * A2[j]);
      *reinterpret_cast<f4 *>(&mapP[tw][ch][p4]) = Pm;
      *reinterpret_cast<f4 *>(&mapH[tw][ch][p4]) = H;
      if (MAPS && p4 == 0) sumd[tw][ch] = sd;
      __syncthreads();
      f4 mine = h;
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        if (w == tw) mine = h;
        const f4 Pw = *reinterpret_cast<const f4 *>(&mapP[w][ch][p4]), Hw = *reinterpret_cast<const f4 *>(&mapH[w][ch][p4]);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = fmaf(Pw[j], h[j], Hw[j]);
        if (MAPS) total += sumd[w][ch];
      }
      run = mine;                              // and h is the one before the next tile
    }
    if constexpr (!MAPS) {
      if (a.states && on && (t - g.s + s0) % SSM_CHUNK<N> == 0 && t + s0 < g.t1)
        *reinterpret_cast<f4 *>(a.states + ((size_t)(chunk0 + (t - g.s + s0) / SSM_CHUNK<N>) * a.D + c) * N + p4) = run;
      float y[4];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const float2 du = step[s0 + s][ch];
        const f4 b = *reinterpret_cast<const f4 *>(&sB[s0 + s][p4]), cv = *reinterpret_cast<const f4 *>(&sC[s0 + s][p4]);
        y[s & 3] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = TW > 1 ? dec[s][j] : __builtin_amdgcn_exp2f(du.x * A2[j]);
          run[j] = fmaf(e, run[j], du.y * b[j]);
          y[s & 3] = fmaf(cv[j], run[j], y[s & 3]);
        }
        if constexpr (L::P == 4) {
          if ((s & 3) == 3) step[s0 + s - 3 + p4 / 4][ch].x = quad_sums(y, p4 / 4);
        } else {
          const float sum = lane_sum<L::P>(y[s & 3]);
          if (p4 == 0) step[s0 + s][ch].x = sum;
        }
      }
      if constexpr (TW == 1) h = run;
    }
    __syncthreads();
    if constexpr (!MAPS) {
      if (valid) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          y[j] = fmaf(skip[j], x[j], step[ls][lc + j].x);
          if (a.z) y[j] *= z[j] * sigmoid(z[j]);
        }
        put(entry<T>(a.y, a.D, t, ls, lcc), y);
      }
    }
  }
  if (tw != 0 || !on) return;
  if constexpr (MAPS) {
    *reinterpret_cast<f4 *>(a.seg_map + ((size_t)g.slot * a.D + c) * N + p4) = h;
    if (p4 == 0) a.seg_sum[(size_t)g.slot * a.D + c] = total;
  } else if (lastseg && a.final_state) {
    *reinterpret_cast<f4 *>(a.final_state + ((size_t)g.n * a.D + c) * N + p4) = h;
  }
}

// The states that the segments of a sequence start from, in order: thread per (channel, 4 states), which loads
// CHAIN_AHEAD maps together.
template <int N> __global__ __launch_bounds__(256) void ssm_chain(SsmArgs a) {
  const int per = a.D * (N / 4), i = blockIdx.x * 256 + threadIdx.x;
  if (i >= per) return;
  const int c = i / (N / 4), p4 = (i % (N / 4)) * 4;
  const f4 A2 = *reinterpret_cast<const f4 *>(a.A + (size_t)c * N + p4) * SSM_LOG2E;
  for (int n = blockIdx.y; n < a.seq.n; n += gridDim.y) {
    const int s = a.seq.begin(n), e = a.seq.end(n), slot = first_slot(a.seq, n, a.seg);
    f4 h{0.f, 0.f, 0.f, 0.f};
    if (a.init) h = *reinterpret_cast<const f4 *>(a.init + ((size_t)n * a.D + c) * N + p4);
    const int maps = e > s ? (e - s - 1) / a.seg : 0;      // of all segments but the last
    for (int k0 = 0; k0 < maps; k0 += CHAIN_AHEAD) {
      f4 H[CHAIN_AHEAD];
      float sd[CHAIN_AHEAD];
#pragma unroll
      for (int k = 0; k < CHAIN_AHEAD; ++k) {
        const size_t at = (size_t)(slot + min(k0 + k, maps - 1)) * a.D + c;
        sd[k] = a.seg_sum[at];
        H[k] = *reinterpret_cast<const f4 *>(a.seg_map + at * N + p4);
      }
#pragma unroll
      for (int k = 0; k < CHAIN_AHEAD; ++k) {
        if (k0 + k >= maps) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = fmaf(__builtin_amdgcn_exp2f(sd[k] * A2[j]), h[j], H[k][j]);
        *reinterpret_cast<f4 *>(a.seg_state + ((size_t)(slot + k0 + k + 1) * a.D + c) * N + p4) = h;
      }
    }
  }
}

// Workgroups of a sequence follow each other, so its number is the same in every lane.
constexpr int STEP_THR = 256;
template <int N> __host__ __device__ int step_blocks(int D) { return (D * (N / 4) + STEP_THR - 1) / STEP_THR; }
template <typename T, int N> __global__ __launch_bounds__(STEP_THR) void ssm_step(SsmArgs a) {
  constexpr int P = N / 4;
  const int per = step_blocks<N>(a.D), n = blockIdx.x / per, i = (blockIdx.x - n * per) * STEP_THR + threadIdx.x;
  const int c = min(i / P, a.D - 1), p4 = i % P * 4;    // whole waves stay for the sum over lanes
  const int64_t row = (int64_t)n * a.D + c;
  const size_t at = (size_t)row * N + p4;
  const f4 h0 = *reinterpret_cast<const f4 *>(a.init + at);
  const f4 A = *reinterpret_cast<const f4 *>(a.A + (size_t)c * N + p4);
  Few<T, 4> B, C;
  Few<T, 1> x, dt, z{};
  fetch(static_cast<const T *>(a.B) + (int64_t)n * a.ldB + p4, B);
  fetch(static_cast<const T *>(a.C) + (int64_t)n * a.ldC + p4, C);
  fetch(static_cast<const T *>(a.x) + (int64_t)n * a.ldx + c, x);
  fetch(static_cast<const T *>(a.dt) + (int64_t)n * a.lddt + c, dt);
  if (a.z) fetch(static_cast<const T *>(a.z) + (int64_t)n * a.ldz + c, z);
  float d = dt[0] + (a.bias ? a.bias[c] : 0.f);
  if (a.softplus) d = softplus(d);
  f4 h;
  float y = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = fmaf(__builtin_amdgcn_exp2f(d * (A[j] * SSM_LOG2E)), h0[j], d * x[0] * B[j]);
    y = fmaf(C[j], h[j], y);
  }
  y = lane_sum<P>(y);
  if (i / P >= a.D) return;
  *reinterpret_cast<f4 *>(a.final_state + at) = h;
  if (p4) return;
  if (a.skip) y = fmaf(a.skip[c], x[0], y);
  if (a.z) y *= z[0] * sigmoid(z[0]);
  static_cast<T *>(a.y)[row] = (T)y;
}

}  // namespace

bool ssm_step_fits(int n, int D, int N) {
  return grid_fits((int64_t)n * (((int64_t)D * N / 4 + STEP_THR - 1) / STEP_THR), STEP_THR);
}

bool ssm_fits(SeqMap seq, int D, int N) {
  const int64_t groups = (D + SSM_FWD_CH - 1) / SSM_FWD_CH;
  const int64_t seg = ssm_segment_fwd(seq, D, N);
  const int64_t slots = seq.cu ? seq.T / seg + seq.n : (int64_t)seq.n * ((seq.T + seg - 1) / seg);
  return slots <= INT32_MAX - 8 && grid_fits(slots * (groups + 7) / 8 * 8 + 8, 1024);
}

size_t ssm_fwd_workspace(SeqMap seq, int D, int N) {
  const int seg = ssm_segment_fwd(seq, D, N);
  if (!ssm_segmented(seq, seg)) return 0;
  const size_t slots = slots_of(seq, seg) + 1;
  return 2 * align16(slots * D * N * sizeof(float)) + align16(slots * D * sizeof(float));
}

template <typename T, int N, int TW, int STEPS> static hipError_t fwd(SsmArgs a, void *ws, hipStream_t s) {
  constexpr int THR = SsmTile<N, SSM_FWD_CH, TW, STEPS>::THR;
  const int groups = (a.D + SSM_FWD_CH - 1) / SSM_FWD_CH;
  const unsigned grid = (unsigned)ssm_grid(groups, slots_of(a.seq, a.seg));
  if (ssm_segmented(a.seq, a.seg)) {
    const size_t states = align16((size_t)(slots_of(a.seq, a.seg) + 1) * a.D * N * sizeof(float));
    a.seg_map = static_cast<float *>(ws);
    a.seg_state = reinterpret_cast<float *>(static_cast<char *>(ws) + states);
    a.seg_sum = reinterpret_cast<float *>(static_cast<char *>(ws) + 2 * states);
    hipLaunchKernelGGL((ssm_fwd<T, N, TW, STEPS, true>), dim3(grid), dim3(THR), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int rows = a.seq.n < 65535 ? a.seq.n : 65535;
    hipLaunchKernelGGL((ssm_chain<N>), dim3((a.D * (N / 4) + 255) / 256, rows), dim3(256), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssm_fwd<T, N, TW, STEPS, false>), dim3(grid), dim3(THR), 0, s, a);
  return hipGetLastError();
}

template <typename T, int N> static hipError_t fwd(SsmArgs a, void *ws, hipStream_t s) {
  a.seg = ssm_segment_fwd(a.seq, a.D, N);
  if (ssm_few_fwd(a.seq, a.seg, a.D)) return fwd<T, N, 128 / N, (N == 64 ? 16 : 8)>(a, ws, s);
  return fwd<T, N, 64 / N, 16>(a, ws, s);
}

hipError_t launch_ssm_fwd(bool bf16, int N, SsmArgs a, void *ws, hipStream_t s) {
  if (N == 16) return bf16 ? fwd<__bf16, 16>(a, ws, s) : fwd<float, 16>(a, ws, s);
  if (N == 32) return bf16 ? fwd<__bf16, 32>(a, ws, s) : fwd<float, 32>(a, ws, s);
  if (N == 64) return bf16 ? fwd<__bf16, 64>(a, ws, s) : fwd<float, 64>(a, ws, s);
  return hipErrorInvalidValue;
}

hipError_t launch_ssm_step(bool bf16, int N, SsmArgs a, hipStream_t s) {
#define FALCON_STEP(N_)                                                                              \
  if (N == N_) {                                                                                     \
    const dim3 grid((unsigned)a.seq.n * step_blocks<N_>(a.D));                                       \
    if (bf16) hipLaunchKernelGGL((ssm_step<__bf16, N_>), grid, dim3(STEP_THR), 0, s, a);             \
    else hipLaunchKernelGGL((ssm_step<float, N_>), grid, dim3(STEP_THR), 0, s, a);                   \
    return hipGetLastError();                                                                        \
  }
  FALCON_STEP(16)
  FALCON_STEP(32)
  FALCON_STEP(64)
#undef FALCON_STEP
  return hipErrorInvalidValue;
}

}  // namespace falcon
