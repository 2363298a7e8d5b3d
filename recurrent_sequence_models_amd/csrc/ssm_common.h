// What the selective state-space scan's kernels share: the layout of a tile, its steps, and the
// slots of a call's segments and chunks.
//
// A wave's lane holds 4 states of one channel: P = N / 4 lanes beside each other make a channel, so a
// sum over the states is one over 4 registers and P neighbouring lanes.  A workgroup owns CH
// channels: WIDE waves lie side by side over them and TW behind each other in time, each
// with STEPS consecutive steps of a tile of TS = STEPS TW.
#pragma once
#include "block_kernels.h"
#include "row_io.h"

namespace falcon {

constexpr int CHAIN_AHEAD = 8;    // segments' maps that are on their way together
constexpr float SSM_LOG2E = 1.44269504088896340736f, SSM_LN2 = 0.69314718055994530942f;

template <int N, int CH_, int TW_, int STEPS_> struct SsmTile {
  static constexpr int CH = CH_, TW = TW_, STEPS = STEPS_, P = N / 4, CW = 64 / P, WIDE = CH / CW, THR = 64 * WIDE * TW;
  static constexpr int TS = TW * STEPS;
  static constexpr int VEC = TS * CH / THR;     // channels of a step that a thread loads: 4, 2 or 1
  static constexpr int BV = TS * N / THR;       // entries of B and C that it loads
  static_assert(WIDE * CW == CH && VEC * THR == TS * CH && BV * THR == TS * N, "a tile is dealt out evenly");
};
// steps between the states that the forward keeps
template <int N> constexpr int SSM_CHUNK = 1024 / N;

// Entries `col` on of token t + row of an array, as scalar base plus 32 bits a lane: t is the same in every lane, and
// token strides are at most 2^24 bytes.
template <typename T> __device__ __forceinline__ const T *entry(const void *p, int64_t ld, int t, int row, int col) {
  const char *base = static_cast<const char *>(p) + (int64_t)t * ld * (int64_t)sizeof(T);
  return reinterpret_cast<const T *>(base + (unsigned)(row * ((int)ld * (int)sizeof(T)) + col * (int)sizeof(T)));
}
template <typename T> __device__ __forceinline__ T *entry(void *p, int64_t ld, int t, int row, int col) {
  char *base = static_cast<char *>(p) + (int64_t)t * ld * (int64_t)sizeof(T);
  return reinterpret_cast<T *>(base + (unsigned)(row * ((int)ld * (int)sizeof(T)) + col * (int)sizeof(T)));
}

// softplus(v) = max(v, 0) + ln(1 + e), e = e^-|v| in (0, 1]; ln(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, and
// atanh(s) = s + s q p(q), q = s^2, with p the cubic that interpolates 1/3 + q/5 + q^2/7 + .. at the Chebyshev nodes of
// [0, 1/9] (off by 2^-25.8 of the logarithm): relative precision however small e is.
__device__ __forceinline__ float softplus(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * SSM_LOG2E);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
  float p = fmaf(q, 0.13425749f, 0.141183099f);
  p = fmaf(p, q, 0.200037803f);
  p = fmaf(p, q, 0.333333202f);
  return fmaxf(v, 0.f) + 2.f * fmaf(p * q, s, s);
}

// The sums over a channel's 4 lanes of 4 values each: lane p gets that of y[p], by two exchanges that halve
// the number of values (9 instructions, where 4 sums of their own take 8 and leave 4 stores).
__device__ __forceinline__ float quad_sums(const float (&y)[4], int p) {
  const bool odd = p & 1, high = p & 2;
  const float u = (odd ? y[1] : y[0]) + dpp_mov<0xB1>(odd ? y[0] : y[1]);
  const float v = (odd ? y[3] : y[2]) + dpp_mov<0xB1>(odd ? y[2] : y[3]);
  return (high ? v : u) + dpp_mov<0x4E>(high ? u : v);
}

// A sequence's part that one workgroup runs over: tokens t0 .. t1 - 1 of sequence n, which begins at s
// and ends at e; `slot` names it among the call's.  Sequence n's segments of `len` tokens
// start at slot begin(n) / len + n, which no two sequences share (floor(a) + ceil(b) <= floor(a + b) + 1);
// sequences of the same length have ceil(T / len) each.
struct Segment { int n, slot, s, e, t0, t1; bool any; };

__device__ __forceinline__ int first_slot(const SeqMap &q, int n, int len) {
  return q.cu ? q.begin(n) / len + n : n * segments_of(q, len);
}
__device__ __forceinline__ Segment find_segment(const SeqMap &q, int len, int slot) {
  Segment g;
  g.slot = slot;
  if (!q.cu) {
    g.n = slot / segments_of(q, len);
  } else {
    int lo = 0, more = q.n;
    while (more > 1) {
      const int half = more >> 1;
      if (first_slot(q, lo + half, len) <= slot) { lo += half; more -= half; } else { more = half; }
    }
    g.n = lo;
  }
  g.s = q.begin(g.n);
  g.e = max(q.end(g.n), g.s);
  const int64_t at = g.s + (int64_t)(slot - first_slot(q, g.n, len)) * len;
  g.t0 = (int)(at < g.e ? at : g.e);
  g.t1 = (int)(at + len < g.e ? at + len : g.e);
  g.any = at >= g.s && at < g.e;
  return g;
}

// The workgroup's segment and channels.  Workgroups are dealt to the 8 dies in turn.  Neighbours in channels share
// cache lines of x and the tiles of B and C, so where there are enough, a die gets an eighth of the channels, of every
// segment (segments differ in length).
struct SsmPlace { int slot, group; bool any; };
constexpr int SSM_DEALT = 64;
__host__ __device__ inline int64_t ssm_grid(int groups, int slots) {
  return groups >= SSM_DEALT ? (int64_t)(groups + 7) / 8 * 8 * slots : (int64_t)groups * slots;
}
__device__ __forceinline__ SsmPlace ssm_place(int groups, int slots) {
  SsmPlace p;
  if (groups >= SSM_DEALT) {
    const int per = (groups + 7) / 8, i = (int)(blockIdx.x / 8);
    p.group = (int)(blockIdx.x % 8) * per + i % per;
    p.slot = i / per;
  } else {
    p.group = (int)(blockIdx.x % groups);
    p.slot = (int)(blockIdx.x / groups);
  }
  p.any = p.group < groups && p.slot < slots;
  return p;
}

}  // namespace falcon
