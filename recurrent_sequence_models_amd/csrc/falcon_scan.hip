// Gated linear recurrence on gfx950: per channel, with lam_t = e^{g_t},
//   h_t = lam_t h_{t-1} + u_t,   u_t = x_t (add) or (1 - lam_t) x_t (mix),
// and its reverse-time adjoint
//   delta_t = dh_t + r_{t+1},  r_t = lam_t delta_t,
//   dx_t = delta_t (times 1 - lam_t),  dg_t = r_t (h_{t-1} [- x_t]),  d init = r at the first step.
//
// Both directions are chains of affine maps of the carried value, y -> A y + H, and
// those compose: (A2, H2) after (A1, H1) is (A1 A2, A2 H1 + H2).  So time is cut three
// times: a thread owns a few consecutive steps of 16 bytes of channels, a workgroup
// CHUNK = 256 steps of one 128-byte column of channels, and the workgroups of a column
// are chained.  Every element is read once and written once: a thread keeps its raw
// inputs in registers between forming its map and replaying its steps from the carry.
//
// The chain of a column.  A workgroup draws its chunk number from the column's ticket
// counter, so the chunks before its own were all drawn by workgroups that already run:
// a wait for them always ends, whatever order the hardware starts workgroups in.  It
// publishes its chunk's map, then waits for the maps of the chunks before it in its
// group of 16 and for the value carried into the group (published by the last chunk of
// the group before), and applies them in order.  The order of operations is fixed, so
// results do not depend on timing.  Groups keep the serial part short: a hop between
// workgroups (store, then another die's load) costs about a microsecond, and one hop
// per chunk would take longer than streaming the chunks.  A published word is 64 bits
// (value and map factor, or value and a mark) written by one atomic store, so no other
// ordering is needed; all ones means "not there yet", which no published word is.
//
// Sequence starts.  The first step of a sequence does not see the carry: its map has
// A = -0, and a map with the sign bit set is applied as y -> H, not as 0 y + H, so an
// infinite or NaN state of one sequence does not reach the next.  Products of decays
// keep the sign: -0 times a decay >= 0 is -0.
//
// Bound: HBM.  Algorithmic bytes: forward 3, backward 5 elements of the input type per
// step and channel.
#include "layer_kernels.h"
#include "mfma_frag.h"

namespace falcon {
namespace {

constexpr int CHUNK = 256;    // steps per workgroup (FALCON_SCAN_CHUNK)
constexpr int LPR = 8;        // lanes side by side in a 128-byte column
constexpr int GROUP = 16;     // chunks whose maps a workgroup applies itself
constexpr unsigned long long EMPTY = ~0ull;

template <typename T> constexpr int CPT = 16 / (int)sizeof(T);   // channels per thread
template <typename T> constexpr int TC = LPR * CPT<T>;           // channels per column

// ---- 16 bytes of channels ----------------------------------------------------
__device__ __forceinline__ void unpack16(const uint4 &u, float (&o)[8]) {
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[2 * j] = __uint_as_float(w[j] << 16);
    o[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack16(const uint4 &u, float (&o)[4]) {
  o[0] = __uint_as_float(u.x); o[1] = __uint_as_float(u.y);
  o[2] = __uint_as_float(u.z); o[3] = __uint_as_float(u.w);
}
// Rounded to nearest even: the one rounding of a result held in bf16.
__device__ __forceinline__ uint4 pack16(const float (&v)[8]) {
  bf8 b;
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = (__bf16)v[j];
  return __builtin_bit_cast(uint4, b);
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4]) {
  return uint4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}
template <int N> __device__ __forceinline__ void load_f32(const float *p, float (&o)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const f4 v = *reinterpret_cast<const f4 *>(p + j);
    o[j] = v[0]; o[j + 1] = v[1]; o[j + 2] = v[2]; o[j + 3] = v[3];
  }
}
template <int N> __device__ __forceinline__ void store_f32(float *p, const float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4) *reinterpret_cast<f4 *>(p + j) = f4{v[j], v[j + 1], v[j + 2], v[j + 3]};
}

// e^g by the hardware's exp2.  Rounding g log2(e) costs |g| 2^-24 relative, which only
// grows where the decay itself has become negligible against 1.
__device__ __forceinline__ float decay(float g) { return __builtin_amdgcn_exp2f(g * 1.44269504088896f); }

// 1 - e^g: the series -(g + g^2/2! + ... + g^7/7!) near 0, where 1 - lam would cancel
// (|g| <= 1/4: the next term is below 2^-28 of the result), else 1 - lam.
__device__ __forceinline__ float one_minus_decay(float g, float lam) {
  float p = 1.f + g * (1.f / 7.f);
  p = 1.f + g * (1.f / 6.f) * p;
  p = 1.f + g * (1.f / 5.f) * p;
  p = 1.f + g * (1.f / 4.f) * p;
  p = 1.f + g * (1.f / 3.f) * p;
  p = 1.f + g * (1.f / 2.f) * p;
  return fabsf(g) <= 0.25f ? -g * p : 1.f - lam;
}

// y after the map (A, H); a set sign of A cuts the carry off.
__device__ __forceinline__ float apply(float A, float H, float y) {
  return (__float_as_uint(A) >> 31) ? H : fmaf(A, y, H);
}

// ---- Published words ---------------------------------------------------------
__device__ __forceinline__ unsigned long long word(float A, float H) {
  unsigned a = __float_as_uint(A);
  if (a == 0xffffffffu) a = 0x7fc00000u;   // a NaN map must not look like an empty word
  return ((unsigned long long)a << 32) | __float_as_uint(H);
}
__device__ __forceinline__ void publish(unsigned long long *p, unsigned long long v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek(const unsigned long long *p) {
  return __hip_atomic_load(const_cast<unsigned long long *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The value carried into the chunk of rank `rank` (its place in the column's chain) for
// one channel: the group's carry, then the maps of the group's earlier chunks in order.
__device__ __forceinline__ float carry_in(const unsigned long long *agg, const unsigned long long *pre, int rank,
                                          int tc) {
  const int g0 = rank & ~(GROUP - 1), j = rank - g0;
  unsigned long long w[GROUP];
  unsigned long long c = 0;
  bool wait;
  do {   // ends: every word waited for belongs to a chunk whose ticket was drawn earlier
    wait = false;
    if (g0) {
      c = peek(pre + (size_t)(rank / GROUP) * tc);
      wait |= c == EMPTY;
    }
#pragma unroll
    for (int i = 0; i < GROUP - 1; ++i)
      if (i < j) {
        w[i] = peek(agg + (size_t)(g0 + i) * tc);
        wait |= w[i] == EMPTY;
      }
    if (wait) __builtin_amdgcn_s_sleep(1);
  } while (wait);
  float y = g0 ? __uint_as_float((unsigned)c) : 0.f;
#pragma unroll
  for (int i = 0; i < GROUP - 1; ++i)
    if (i < j) y = apply(__uint_as_float((unsigned)(w[i] >> 32)), __uint_as_float((unsigned)w[i]), y);
  return y;
}

// ---- Sequences ---------------------------------------------------------------
// The sequence that holds token t: the largest n < N with cu[n] <= t (cu[0] if none).
__device__ __forceinline__ int seq_of(const int *cu, int N, int t) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Which of a thread's steps t0 .. t0 + SEG - 1 are the first or last of a sequence, and
// how many are inside one (the rest are behind the last sequence or the time axis).
struct Marks { unsigned first, last; int valid; };

template <int SEG> __device__ __forceinline__ Marks marks_of(const ScanArgs &a, int t0) {
  Marks m{0, 0, 0};
  if (!a.cu) {
    m.valid = min(max(a.T - t0, 0), SEG);
    if (t0 == 0) m.first = 1;
    if (a.T - 1 >= t0 && a.T - 1 < t0 + SEG) m.last = 1u << (a.T - 1 - t0);
    return m;
  }
  const int end = min(a.cu[a.nseq], a.T);
  m.valid = min(max(end - t0, 0), SEG);
  if (m.valid == 0) return m;
  int n = seq_of(a.cu, a.nseq, t0);
  if (a.cu[n] == t0) m.first = 1;
  for (; n < a.nseq; ++n) {      // walk the sequence ends inside the steps
    const int e = a.cu[n + 1];
    if (e > t0 + SEG) break;
    if (e > t0) {
      m.last |= 1u << (e - 1 - t0);
      if (e < end && e < t0 + SEG) m.first |= 1u << (e - t0);
    }
  }
  return m;
}
// The sequence of step t of this row (batch rows are their own sequences).
__device__ __forceinline__ int seq_at(const ScanArgs &a, int row, int t) {
  return a.cu ? seq_of(a.cu, a.nseq, t) : row;
}

struct Place { int row, rank, c0; size_t col; };

// Column (batch row, 128-byte column of channels) and rank in its chain.
template <typename T> __device__ __forceinline__ Place place(const ScanArgs &a) {
  const int tiles = (a.D + TC<T> - 1) / TC<T>;
  const unsigned ncol = (unsigned)a.rows * tiles;
  const unsigned col = blockIdx.x % ncol;
  Place p;
  p.col = col;
  p.row = col / tiles;
  p.c0 = (col - p.row * tiles) * TC<T>;
  p.rank = 0;
  if (a.NC > 1) {
    __shared__ unsigned drawn;
    // counters start at all ones, like every word of the workspace
    if (threadIdx.x == 0)
      drawn = __hip_atomic_fetch_add(a.ticket + col, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
    __syncthreads();
    p.rank = __builtin_amdgcn_readfirstlane((int)drawn);
  }
  return p;
}

// An empty sequence ends where it began: its rows are copied (zeros without a source).
template <int N>
__device__ __forceinline__ void copy_empty(const ScanArgs &a, const float *from, float *to, int rank, int grp, int ngrp,
                                           int ch) {
  if (!a.cu || !to || ch >= a.D) return;
  for (int n = rank * ngrp + grp; n < a.nseq; n += a.NC * ngrp) {
    if (a.cu[n] != a.cu[n + 1]) continue;
    float v[N] = {};
    if (from) load_f32<N>(from + (size_t)n * a.D + ch, v);
    store_f32<N>(to + (size_t)n * a.D + ch, v);
  }
}

// ---- Forward -----------------------------------------------------------------
// 256 threads: 32 groups of 8 lanes, each group 8 steps.
constexpr int FSEG = 8, FGRP = CHUNK / FSEG, FTHR = FGRP * LPR;

template <typename T, bool MIX> __global__ __launch_bounds__(FTHR) void scan_fwd(ScanArgs a) {
  constexpr int C = CPT<T>, W = TC<T>;
  __shared__ __align__(16) float sA[FGRP][W], sH[FGRP][W];   // group maps; sH then holds the groups' carries
  const Place p = place<T>(a);
  const int tid = threadIdx.x, grp = tid / LPR, cl = (tid % LPR) * C, ch = p.c0 + cl;
  const int t0 = p.rank * CHUNK + grp * FSEG;
  const bool on = ch < a.D;
  Marks m = marks_of<FSEG>(a, t0);
  if (!on) m = Marks{0, 0, 0};
  const T *x = static_cast<const T *>(a.x) + ((size_t)p.row * a.T + t0) * a.D + ch;
  const T *g = static_cast<const T *>(a.g) + ((size_t)p.row * a.T + t0) * a.D + ch;
  uint4 xr[FSEG], gr[FSEG];
#pragma unroll
  for (int i = 0; i < FSEG; ++i) {   // steps outside are x = 0, g = 0: the identity map
    xr[i] = gr[i] = uint4{0, 0, 0, 0};
    if (i < m.valid) {
      xr[i] = *reinterpret_cast<const uint4 *>(x + (size_t)i * a.D);
      gr[i] = *reinterpret_cast<const uint4 *>(g + (size_t)i * a.D);
    }
  }
  copy_empty<C>(a, a.init, a.final_state, p.rank, grp, FGRP, ch);

  // this thread's map; h0 keeps the initial state of the last sequence that starts here (another
  // workgroup may write its final state, which may be the same memory, before the replay below)
  float A[C], H[C], h0[C] = {};
#pragma unroll
  for (int c = 0; c < C; ++c) { A[c] = 1.f; H[c] = 0.f; }
#pragma unroll
  for (int i = 0; i < FSEG; ++i) {
    if ((m.first >> i) & 1) {
      if (a.init) load_f32<C>(a.init + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, h0);
#pragma unroll
      for (int c = 0; c < C; ++c) { A[c] = -0.f; H[c] = h0[c]; }
    }
    float xv[C], gv[C];
    unpack16(xr[i], xv);
    unpack16(gr[i], gv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      const float u = MIX ? one_minus_decay(gv[c], lam) * xv[c] : xv[c];
      A[c] *= lam;
      H[c] = fmaf(lam, H[c], u);
    }
  }
  store_f32<C>(&sA[grp][cl], A);
  store_f32<C>(&sH[grp][cl], H);
  __syncthreads();
  if (tid < W) {   // one lane a channel: the chunk's map, the carry, the groups' carries
    float At = 1.f, Ht = 0.f;
#pragma unroll 8
    for (int q = 0; q < FGRP; ++q) {
      Ht = apply(sA[q][tid], sH[q][tid], Ht);
      At *= sA[q][tid];
    }
    float y = 0.f;
    if (a.NC > 1) {
      const int ng = (a.NC + GROUP - 1) / GROUP;
      unsigned long long *agg = a.agg + p.col * a.NC * W + tid, *pre = a.pre + p.col * ng * W + tid;
      if (p.rank + 1 < a.NC) publish(agg + (size_t)p.rank * W, word(At, Ht));
      y = carry_in(agg, pre, p.rank, W);
      if (p.rank % GROUP == GROUP - 1 && p.rank + 1 < a.NC)
        publish(pre + (size_t)(p.rank / GROUP + 1) * W, word(0.f, apply(At, Ht, y)));
    }
    if (a.states && p.c0 + tid < a.D)
      a.states[((size_t)p.row * a.NC + p.rank) * a.D + p.c0 + tid] = apply(At, Ht, y);
#pragma unroll 8
    for (int q = 0; q < FGRP; ++q) {
      const float Hq = sH[q][tid];
      sH[q][tid] = y;
      y = apply(sA[q][tid], Hq, y);
    }
  }
  __syncthreads();
  float h[C];
  load_f32<C>(&sH[grp][cl], h);
  T *out = static_cast<T *>(a.h) + ((size_t)p.row * a.T + t0) * a.D + ch;
#pragma unroll
  for (int i = 0; i < FSEG; ++i) {
    if (i >= m.valid) break;
    if ((m.first >> i) & 1) {
      if (m.first >> (i + 1)) {   // a sequence inside these steps: read again, this thread alone writes its end
#pragma unroll
        for (int c = 0; c < C; ++c) h[c] = 0.f;
        if (a.init) load_f32<C>(a.init + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, h);
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) h[c] = h0[c];
      }
    }
    float xv[C], gv[C];
    unpack16(xr[i], xv);
    unpack16(gr[i], gv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      const float u = MIX ? one_minus_decay(gv[c], lam) * xv[c] : xv[c];
      h[c] = fmaf(lam, h[c], u);
    }
    *reinterpret_cast<uint4 *>(out + (size_t)i * a.D) = pack16(h);
    if (((m.last >> i) & 1) && a.final_state)
      store_f32<C>(a.final_state + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, h);
  }
}

// ---- Backward ----------------------------------------------------------------
// 512 threads: 64 groups of 8 lanes, each group 4 steps (a step has three inputs, and its
// incoming state is kept from the forward replay: half the forward's steps per thread).
// The states of the forward's chunks give the state entering a chunk; only the reverse
// direction is chained.
constexpr int BSEG = 4, BGRP = CHUNK / BSEG, BTHR = BGRP * LPR;

template <typename T, bool MIX> __global__ __launch_bounds__(BTHR) void scan_bwd(ScanArgs a) {
  constexpr int C = CPT<T>, W = TC<T>;
  __shared__ __align__(16) float sA[BGRP][W], sH[BGRP][W];   // forward maps
  __shared__ __align__(16) float sR[BGRP][W], sQ[BGRP][W];   // reverse maps
  const Place p = place<T>(a);
  const int chunk = a.NC - 1 - p.rank;
  const int tid = threadIdx.x, grp = tid / LPR, cl = (tid % LPR) * C, ch = p.c0 + cl;
  const int t0 = chunk * CHUNK + grp * BSEG;
  const bool on = ch < a.D;
  Marks m = marks_of<BSEG>(a, t0);
  if (!on) m = Marks{0, 0, 0};
  const size_t at = ((size_t)p.row * a.T + t0) * a.D + ch;
  const T *x = static_cast<const T *>(a.x) + at, *g = static_cast<const T *>(a.g) + at;
  const T *dh = static_cast<const T *>(a.dh) + at;
  uint4 xr[BSEG], gr[BSEG], dr[BSEG];
#pragma unroll
  for (int i = 0; i < BSEG; ++i) {
    xr[i] = gr[i] = dr[i] = uint4{0, 0, 0, 0};
    if (i < m.valid) {
      xr[i] = *reinterpret_cast<const uint4 *>(x + (size_t)i * a.D);
      gr[i] = *reinterpret_cast<const uint4 *>(g + (size_t)i * a.D);
      dr[i] = *reinterpret_cast<const uint4 *>(dh + (size_t)i * a.D);
    }
  }
  copy_empty<C>(a, a.d_final, a.d_init, p.rank, grp, BGRP, ch);

  float A[C], H[C];
#pragma unroll
  for (int c = 0; c < C; ++c) { A[c] = 1.f; H[c] = 0.f; }
#pragma unroll
  for (int i = 0; i < BSEG; ++i) {
    if ((m.first >> i) & 1) {
      float h0[C] = {};
      if (a.init) load_f32<C>(a.init + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, h0);
#pragma unroll
      for (int c = 0; c < C; ++c) { A[c] = -0.f; H[c] = h0[c]; }
    }
    float xv[C], gv[C];
    unpack16(xr[i], xv);
    unpack16(gr[i], gv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      A[c] *= lam;
      H[c] = fmaf(lam, H[c], MIX ? one_minus_decay(gv[c], lam) * xv[c] : xv[c]);
    }
  }
  store_f32<C>(&sA[grp][cl], A);
  store_f32<C>(&sH[grp][cl], H);
  // the reverse map of these steps: r_{t+1} of the last to r_t of the first
#pragma unroll
  for (int c = 0; c < C; ++c) { A[c] = 1.f; H[c] = 0.f; }
#pragma unroll
  for (int i = BSEG - 1; i >= 0; --i) {
    if ((m.last >> i) & 1) {
      float d0[C] = {};
      if (a.d_final) load_f32<C>(a.d_final + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, d0);
#pragma unroll
      for (int c = 0; c < C; ++c) { A[c] = -0.f; H[c] = d0[c]; }
    }
    float gv[C], dv[C];
    unpack16(gr[i], gv);
    unpack16(dr[i], dv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      A[c] *= lam;
      H[c] = lam * (dv[c] + H[c]);
    }
  }
  store_f32<C>(&sR[grp][cl], A);
  store_f32<C>(&sQ[grp][cl], H);
  __syncthreads();
  if (tid < W) {                          // one wave: the reverse chain
    float At = 1.f, Ht = 0.f;
#pragma unroll 8
    for (int q = BGRP - 1; q >= 0; --q) {
      Ht = apply(sR[q][tid], sQ[q][tid], Ht);
      At *= sR[q][tid];
    }
    float y = 0.f;
    if (a.NC > 1) {
      const int ng = (a.NC + GROUP - 1) / GROUP;
      unsigned long long *agg = a.agg + p.col * a.NC * W + tid, *pre = a.pre + p.col * ng * W + tid;
      if (p.rank + 1 < a.NC) publish(agg + (size_t)p.rank * W, word(At, Ht));
      y = carry_in(agg, pre, p.rank, W);
      if (p.rank % GROUP == GROUP - 1 && p.rank + 1 < a.NC)
        publish(pre + (size_t)(p.rank / GROUP + 1) * W, word(0.f, apply(At, Ht, y)));
    }
#pragma unroll 8
    for (int q = BGRP - 1; q >= 0; --q) {
      const float Hq = sQ[q][tid];
      sQ[q][tid] = y;
      y = apply(sR[q][tid], Hq, y);
    }
  } else if (tid >= 64 && tid < 64 + W) {  // another wave: the states entering the groups
    const int l = tid - 64;
    float y = 0.f;
    if (chunk > 0 && p.c0 + l < a.D) y = a.states[((size_t)p.row * a.NC + chunk - 1) * a.D + p.c0 + l];
#pragma unroll 8
    for (int q = 0; q < BGRP; ++q) {
      const float Hq = sH[q][l];
      sH[q][l] = y;
      y = apply(sA[q][l], Hq, y);
    }
  }
  __syncthreads();
  if (m.valid == 0) return;
  float h[C], hp[BSEG][C];                // hp: the state entering each step
  load_f32<C>(&sH[grp][cl], h);
#pragma unroll
  for (int i = 0; i < BSEG; ++i) {
    if ((m.first >> i) & 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = 0.f;
      if (a.init) load_f32<C>(a.init + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, h);
    }
    float xv[C], gv[C];
    unpack16(xr[i], xv);
    unpack16(gr[i], gv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      hp[i][c] = h[c];
      h[c] = fmaf(lam, h[c], MIX ? one_minus_decay(gv[c], lam) * xv[c] : xv[c]);
    }
  }
  float r[C];
  load_f32<C>(&sQ[grp][cl], r);
  T *dx = static_cast<T *>(a.dx) + at, *dg = static_cast<T *>(a.dg) + at;
#pragma unroll
  for (int i = BSEG - 1; i >= 0; --i) {
    if (i >= m.valid) continue;
    if ((m.last >> i) & 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) r[c] = 0.f;
      if (a.d_final) load_f32<C>(a.d_final + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, r);
    }
    float xv[C], gv[C], dv[C], ox[C], og[C];
    unpack16(xr[i], xv);
    unpack16(gr[i], gv);
    unpack16(dr[i], dv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      const float delta = dv[c] + r[c];
      r[c] = lam * delta;
      ox[c] = MIX ? one_minus_decay(gv[c], lam) * delta : delta;
      og[c] = r[c] * (MIX ? hp[i][c] - xv[c] : hp[i][c]);
    }
    *reinterpret_cast<uint4 *>(dx + (size_t)i * a.D) = pack16(ox);
    *reinterpret_cast<uint4 *>(dg + (size_t)i * a.D) = pack16(og);
    if (((m.first >> i) & 1) && a.d_init)
      store_f32<C>(a.d_init + (size_t)seq_at(a, p.row, t0 + i) * a.D + ch, r);
  }
}

// ---- One step ----------------------------------------------------------------
// state <- lam state + u in place; one thread per 16 bytes of x.
template <typename T, bool MIX>
__global__ __launch_bounds__(256) void scan_step(const T *x, const T *g, float *state, T *h, size_t n) {
  constexpr int C = CPT<T>;
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * C;
  if (i >= n) return;
  float xv[C], gv[C], s[C];
  unpack16(*reinterpret_cast<const uint4 *>(x + i), xv);
  unpack16(*reinterpret_cast<const uint4 *>(g + i), gv);
  load_f32<C>(state + i, s);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float lam = decay(gv[c]);
    s[c] = fmaf(lam, s[c], MIX ? one_minus_decay(gv[c], lam) * xv[c] : xv[c]);
  }
  store_f32<C>(state + i, s);
  *reinterpret_cast<uint4 *>(h + i) = pack16(s);
}

__global__ __launch_bounds__(256) void fill_ones(uint4 *p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
    p[i] = uint4{~0u, ~0u, ~0u, ~0u};
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Byte sizes of the workspace's three arrays.
struct Layout { size_t ticket, agg, pre; };
Layout layout(bool bf16, int rows, int T, int D) {
  const size_t tc = bf16 ? TC<__bf16> : TC<float>;
  const size_t nc = ((size_t)T + CHUNK - 1) / CHUNK, cols = (size_t)rows * ((D + tc - 1) / tc);
  if (nc <= 1) return Layout{0, 0, 0};
  return Layout{up16(cols * 4), cols * nc * tc * 8, cols * ((nc + GROUP - 1) / GROUP) * tc * 8};
}

// Lays the workspace out, fills it, and gives the grid size (0: more workgroups than a grid holds).
hipError_t prepare(bool bf16, ScanArgs &a, void *ws, unsigned &grid, hipStream_t s) {
  const int tc = bf16 ? TC<__bf16> : TC<float>;
  a.NC = (a.T + CHUNK - 1) / CHUNK;
  const size_t blocks = (size_t)a.rows * ((a.D + tc - 1) / tc) * a.NC;
  if (blocks > 0x7fffffffu) return hipErrorInvalidValue;
  grid = (unsigned)blocks;
  if (a.NC == 1) return hipSuccess;
  const Layout l = layout(bf16, a.rows, a.T, a.D);
  unsigned char *p = static_cast<unsigned char *>(ws);
  a.ticket = reinterpret_cast<unsigned int *>(p);
  a.agg = reinterpret_cast<unsigned long long *>(p + l.ticket);
  a.pre = reinterpret_cast<unsigned long long *>(p + l.ticket + l.agg);
  const size_t n16 = (l.ticket + l.agg + l.pre) / 16;
  const unsigned nb = (unsigned)(n16 / 256 + 1 < 2048 ? n16 / 256 + 1 : 2048);
  hipLaunchKernelGGL(fill_ones, dim3(nb), dim3(256), 0, s, static_cast<uint4 *>(ws), n16);
  return hipGetLastError();
}

}  // namespace

size_t scan_workspace(bool bf16, int rows, int T, int D) {
  const Layout l = layout(bf16, rows, T, D);
  return l.ticket + l.agg + l.pre;
}

#define FALCON_SCAN_LAUNCH(KERNEL, THREADS)                                                                \
  unsigned grid = 0;                                                                                       \
  const hipError_t e = prepare(bf16, a, ws, grid, s);                                                      \
  if (e != hipSuccess) return e;                                                                           \
  if (bf16 && mix) hipLaunchKernelGGL((KERNEL<__bf16, true>), dim3(grid), dim3(THREADS), 0, s, a);         \
  else if (bf16) hipLaunchKernelGGL((KERNEL<__bf16, false>), dim3(grid), dim3(THREADS), 0, s, a);          \
  else if (mix) hipLaunchKernelGGL((KERNEL<float, true>), dim3(grid), dim3(THREADS), 0, s, a);             \
  else hipLaunchKernelGGL((KERNEL<float, false>), dim3(grid), dim3(THREADS), 0, s, a);                     \
  return hipGetLastError();

hipError_t launch_scan_fwd(bool bf16, bool mix, ScanArgs a, void *ws, hipStream_t s) {
  FALCON_SCAN_LAUNCH(scan_fwd, FTHR)
}
hipError_t launch_scan_bwd(bool bf16, bool mix, ScanArgs a, void *ws, hipStream_t s) {
  FALCON_SCAN_LAUNCH(scan_bwd, BTHR)
}
#undef FALCON_SCAN_LAUNCH

hipError_t launch_scan_step(bool bf16, bool mix, const void *x, const void *g, float *state, void *h, size_t n,
                            hipStream_t s) {
  const size_t blocks = (n / (bf16 ? 8 : 4) + 255) / 256;
  if (blocks > 0x7fffffffu) return hipErrorInvalidValue;
#define FALCON_STEP1(T_, M_)                                                                                    \
  hipLaunchKernelGGL((scan_step<T_, M_>), dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const T_ *>(x),   \
                     static_cast<const T_ *>(g), state, static_cast<T_ *>(h), n)
  if (bf16 && mix) FALCON_STEP1(__bf16, true);
  else if (bf16) FALCON_STEP1(__bf16, false);
  else if (mix) FALCON_STEP1(float, true);
  else FALCON_STEP1(float, false);
#undef FALCON_STEP1
  return hipGetLastError();
}

}  // namespace falcon
