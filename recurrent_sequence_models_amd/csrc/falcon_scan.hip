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
// infinite or NaN state of one sequence does not reach the next.  Products with decays
// (>= 0) keep the sign, and joining maps sets it where either map's is.
//
// Bound: HBM, with algorithmic bytes of 3 (forward) and 5 (backward) elements of the input type
// per step and channel, and for bf16 the vector unit close behind.  Measured, where a plain
// copy moves 5.1 TB/s:
//   64 x 256 x 2048 bf16, one chunk a sequence: forward 39.8 us (5.1 TB/s), backward 75 us (4.5)
//   65536 x 2048 bf16: forward 183 us (4.4 TB/s); 9001 x 2048 fp32, 13 sequences: 55 to 60 us (3.7 to 4.1)
//   8 x 2048 x 768 bf16, mix: forward 19.5 us (3.9 TB/s), and 2 us to clear the workspace
//   4 x 4096 x 768 bf16, mix: backward 33 us (3.8 TB/s; the vector unit is busy with the decay and
//   1 - lam, formed again where the registers to keep them are the second workgroup's of a
//   compute unit: 45 us without that one)
// A chunk waits for those before it: with few chunks a column (the 768-wide cases) that
// latency is the rest.
#include "layer_kernels.h"
#include "mfma_frag.h"

namespace falcon {
namespace {

constexpr int CHUNK = 256;    // steps per workgroup (FALCON_SCAN_CHUNK)
constexpr int LPR = 8;        // lanes side by side in a 128-byte column
constexpr int GROUP = 16;     // chunks whose maps a workgroup applies itself
constexpr unsigned long long EMPTY = ~0ull;

typedef unsigned int u4 __attribute__((ext_vector_type(4)));   // 16 bytes of channels, in registers

template <typename T> constexpr int CPT = 16 / (int)sizeof(T);   // channels per thread
template <typename T> constexpr int TC = LPR * CPT<T>;           // channels per column

// ---- 16 bytes of channels ----------------------------------------------------
__device__ __forceinline__ void unpack16(const u4 &u, float (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[2 * j] = __uint_as_float(u[j] << 16);
    o[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack16(const u4 &u, float (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = __uint_as_float(u[j]);
}
// Rounded to nearest even: the one rounding of a result held in bf16.
__device__ __forceinline__ u4 pack16(const float (&v)[8]) {
  bf8 b;
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = (__bf16)v[j];
  return __builtin_bit_cast(u4, b);
}
__device__ __forceinline__ u4 pack16(const float (&v)[4]) {
  return u4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
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

// 1 - e^g: the series -g (1 + g / 2! + ... + g^5 / 6!) near 0, where 1 - lam would cancel
// (|g| <= 1/8: the next term is 2^-30 of the result), else 1 - lam (off by 2^-22 at most).
__device__ __forceinline__ float one_minus_decay(float g, float lam) {
  float p = fmaf(g, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(p, g, 1.f / 24.f);
  p = fmaf(p, g, 1.f / 6.f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g, 1.f);
  return fabsf(g) <= 0.125f ? -g * p : 1.f - lam;
}

// The product of two maps' factors; the sign is set where either's is (-0 times -0 would clear it).
__device__ __forceinline__ float join(float A, float B) {
  return __uint_as_float(__float_as_uint(A * B) | ((__float_as_uint(A) | __float_as_uint(B)) & 0x80000000u));
}
// y after the map (A, H); a set sign of A cuts the carry off.
__device__ __forceinline__ float apply(float A, float H, float y) {
  return (__float_as_uint(A) >> 31) ? H : fmaf(A, y, H);
}

// ---- Published words ---------------------------------------------------------
__device__ __forceinline__ unsigned long long word(float A, float H) {
  unsigned a = __float_as_uint(A);
  if (a == 0xffffffffu) a = 0xffc00000u;   // a NaN map must not look like an empty word; its sign still cuts the carry off
  return ((unsigned long long)a << 32) | __float_as_uint(H);
}
__device__ __forceinline__ void publish(unsigned long long *p, unsigned long long v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek(const unsigned long long *p) {
  return __hip_atomic_load(const_cast<unsigned long long *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---- Sequences ---------------------------------------------------------------
// The sequence that holds token t: the largest n < N with cu[n] <= t (0 if none).
__device__ __forceinline__ int seq_of(const int *cu, int N, int t) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The offsets as a wave reads them while it places its steps: up to 63 sequences in one register
// (lane i holds cu[i], loaded before anything else is waited for), more from memory.  Every
// lane of the wave calls them.
struct Offsets {
  const int *cu;
  int N, reg;
  __device__ __forceinline__ Offsets(const ScanArgs &a) : cu(a.cu), N(a.nseq), reg(0) {
    if (cu && N < 64) reg = cu[min((int)(threadIdx.x & 63), N)];
  }
  __device__ __forceinline__ int at(int i) const { return N < 64 ? __shfl(reg, i) : cu[i]; }
  __device__ __forceinline__ int last() const { return N < 64 ? __builtin_amdgcn_readlane(reg, N) : cu[N]; }
  // the sequence that holds token t, the same t in every lane: 64 places at a time
  __device__ __forceinline__ int seq_of(int t) const {
    const int lane = threadIdx.x & 63;
    if (N < 64) return max((int)__popcll(__ballot(lane < N && reg <= t)) - 1, 0);
    int lo = 0, len = N;
    while (len > 1) {
      const int step = (len + 63) / 64, at = lane * step;
      const int before = __popcll(__ballot(at < len && cu[lo + min(at, len - 1)] <= t));
      const int skip = max(before - 1, 0) * step;
      lo += skip;
      len = min(step, len - skip);
    }
    return lo;
  }
};

// Which of a thread's steps t0 .. t0 + SEG - 1 are the first or last of a packed sequence.
// (Batch rows begin and end with the chain: the carry of rank 0 and the chain's result.)
struct Marks { unsigned first, last; };

template <int SEG> __device__ __forceinline__ Marks marks_of(const Offsets &cu, int t0, int end) {
  Marks m{0, 0};
  int n = cu.seq_of(__builtin_amdgcn_readfirstlane(t0));   // of the wave's first step, then of this thread's
  bool more = true;
  while (__any(more)) {
    const int e = cu.at(min(n + 1, cu.N));
    more = n + 1 < cu.N && e <= t0;
    n += more;
  }
  const bool in = t0 < end;
  if (cu.at(n) == t0 && in) m.first = 1;
  more = in;
  while (__any(more)) {          // the sequence ends inside the steps
    const int e = cu.at(min(n + 1, cu.N));
    more = more && n < cu.N && e <= t0 + SEG;
    if (more && e > t0) {
      m.last |= 1u << (e - 1 - t0);
      if (e < end && e < t0 + SEG) m.first |= 1u << (e - t0);
    }
    n += more;
  }
  return m;
}
// The row of a [nseq, D] array of the packed sequence of token t; zeros without the array.
template <int N>
__device__ __forceinline__ void load_seq(const ScanArgs &a, const float *p, int t, int ch, float (&o)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) o[c] = 0.f;
  if (p) load_f32<N>(p + (size_t)seq_of(a.cu, a.nseq, t) * a.D + ch, o);
}
template <int N>
__device__ __forceinline__ void store_seq(const ScanArgs &a, float *p, int t, int ch, const float (&v)[N]) {
  if (p) store_f32<N>(p + (size_t)seq_of(a.cu, a.nseq, t) * a.D + ch, v);
}
// An empty sequence ends where it began: its rows are copied (zeros without a source).
template <int N>
__device__ __forceinline__ void copy_empty(const ScanArgs &a, const float *from, float *to, int rank, int grp, int ngrp,
                                           int ch) {
  if (!to || ch >= a.D) return;
  for (int n = rank * ngrp + grp; n < a.nseq; n += a.NC * ngrp) {
    if (a.cu[n] != a.cu[n + 1]) continue;
    float v[N] = {};
    if (from) load_f32<N>(from + (size_t)n * a.D + ch, v);
    store_f32<N>(to + (size_t)n * a.D + ch, v);
  }
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

// A thread's steps: 16 bytes of channels at each of SEG tokens from t0.  Tokens past `end`
// and channels past D read another place of the same array and become zeros, which as x
// (dh) and log decay are the identity map.  The loads are unconditional, so that all of
// them are in flight at once.
// Addresses are the chunk's (scalar) plus 32 bits a thread: a chunk of the widest rows,
// 2^20 channels, is 2^30 bytes.
template <typename T, int SEG> struct Steps {
  size_t base;         // the chunk's first element
  int t, most, n;      // the thread's first step and the last one of the array, counted in the chunk; its valid steps
  unsigned D, c;
  __device__ __forceinline__ Steps(const ScanArgs &a, int row, int chunk, int grp, int end, int ch) {
    base = ((size_t)row * a.T + (size_t)chunk * CHUNK) * a.D;
    t = grp * SEG;
    most = a.T - 1 - chunk * CHUNK;
    n = ch < a.D ? end - chunk * CHUNK - t : 0;
    D = a.D;
    c = min(ch, a.D - CPT<T>);
  }
  __device__ __forceinline__ unsigned at(int i) const { return (unsigned)min(t + i, most) * D + c; }
  __device__ __forceinline__ void load(const void *p, u4 (&v)[SEG]) const {
    const T *q = static_cast<const T *>(p) + base;
#pragma unroll
    for (int i = 0; i < SEG; ++i) v[i] = *reinterpret_cast<const u4 *>(q + at(i));
  }
  __device__ __forceinline__ void store(void *p, int i, const u4 &v) const {
    if (i < n) *reinterpret_cast<u4 *>(static_cast<T *>(p) + base + at(i)) = v;
  }
  __device__ __forceinline__ void mask(u4 (&v)[SEG]) const {
#pragma unroll
    for (int i = 0; i < SEG; ++i) v[i] = i < n ? v[i] : u4{0, 0, 0, 0};
  }
};

// Makes raw inputs opaque to the compiler, which otherwise keeps every step's decay and input
// in fp32 from one pass over the steps to the next (4 times the registers of the bf16 inputs).
template <int N> __device__ __forceinline__ void forget(u4 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

// lam and u of one step's channels.
template <bool MIX, int C>
__device__ __forceinline__ void step_of(const u4 &x, const u4 &g, float (&lam)[C], float (&u)[C]) {
  float gv[C];
  unpack16(x, u);
  unpack16(g, gv);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    lam[c] = decay(gv[c]);
    if (MIX) u[c] *= one_minus_decay(gv[c], lam[c]);
  }
}

// ---- A chunk's scan -----------------------------------------------------------
// 512 threads: 64 groups of 8 lanes, each group 4 steps; a wave's 8 groups are neighbours
// in time.  Groups, waves and chunks are scanned in turn, 8, 8 and at most 15 maps one
// after the other (a single wave over all 64 groups took 0.8 us of every workgroup's time,
// twice).  2 or 8 steps a thread, and chunks of 128, were no faster.
constexpr int SEG = 4, GRPS = CHUNK / SEG, THR = GRPS * LPR, WAVES = THR / 64, GPW = GRPS / WAVES;

template <int W> struct Maps {
  float A[GRPS][W], H[GRPS][W];          // the groups' maps; H then holds the values carried into them
  float wA[WAVES][W], wH[WAVES][W];      // the waves' maps
};
struct Map { float A, H; };
template <int W> using Words = unsigned long long[GROUP][W];   // words read from the column's chain

// All of these run one lane a channel (lanes < W), in time order or (REV) against it; every
// thread of the workgroup calls them.

// The map of this wave's groups, from the groups' maps that its lanes wrote.
template <int W, bool REV> __device__ __forceinline__ void wave_map(Maps<W> &s) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's maps are in LDS
  if (lane >= W) return;
  float A = 1.f, H = 0.f;
#pragma unroll
  for (int i = 0; i < GPW; ++i) {
    const int q = wave * GPW + (REV ? GPW - 1 - i : i);
    H = apply(s.A[q][lane], s.H[q][lane], H);
    A = join(A, s.A[q][lane]);
  }
  s.wA[wave][lane] = A;
  s.wH[wave][lane] = H;
}
// (A barrier later:) the chunk's map.
template <int W, bool REV> __device__ __forceinline__ Map chunk_map(const Maps<W> &s) {
  const int lane = threadIdx.x & 63;
  Map m{1.f, 0.f};
  if (lane < W)
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const int w = REV ? WAVES - 1 - i : i;
      m.H = apply(s.wA[w][lane], s.wH[w][lane], m.H);
      m.A = join(m.A, s.wA[w][lane]);
    }
  return m;
}
// The values carried into the groups (to s.H), from the one carried into the chunk.
template <int W, bool REV> __device__ __forceinline__ void spread(Maps<W> &s, float y) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane < W) {
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const int w = REV ? WAVES - 1 - i : i;
      const float z = apply(s.wA[w][lane], s.wH[w][lane], y);
      if (REV ? w > wave : w < wave) y = z;
    }
#pragma unroll
    for (int i = 0; i < GPW; ++i) {
      const int q = wave * GPW + (REV ? GPW - 1 - i : i);
      const float H = s.H[q][lane];
      s.H[q][lane] = y;
      y = apply(s.A[q][lane], H, y);
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's carries are in LDS
}

// The chain of a column's chunks (NC > 1).  The chunk of rank `rank` publishes its map; rank 0
// also publishes *first, the value carried into it, which it alone reads, since its memory may
// be where the chain's result goes.
template <int W> struct Chain {
  unsigned long long *agg, *pre;         // this lane's channel: the chunks' maps, the groups' carries
  int rank, grp, j, NC;                  // j: place in the group of chunks
  __device__ __forceinline__ Chain(const ScanArgs &a, size_t col, int rank) : rank(rank), NC(a.NC) {
    const int lane = threadIdx.x & 63, ng = (a.NC + GROUP - 1) / GROUP;
    grp = rank / GROUP;
    j = rank % GROUP;
    agg = a.agg + col * a.NC * W + lane;
    pre = a.pre + col * ng * W + lane;
  }
  __device__ __forceinline__ void give(const Map &m, const float *first) const {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (wave || lane >= W) return;
    if (rank + 1 < NC) publish(agg + (size_t)rank * W, word(m.A, m.H));
    if (rank == 0) publish(pre, word(0.f, first ? first[lane] : 0.f));
  }
  // Every wave reads two words: the maps of the group's chunks before this one, and (word 15) the
  // value carried into the group.
  __device__ __forceinline__ void take(Words<W> &words) const {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane >= W) return;
#pragma unroll
    for (int k = 2 * wave; k < 2 * wave + 2; ++k) {
      if (k >= j && k < GROUP - 1) continue;
      const unsigned long long *p = k == GROUP - 1 ? pre + (size_t)grp * W : agg + (size_t)(grp * GROUP + k) * W;
      unsigned long long v;
      // ends: the word is published by a chunk whose ticket was drawn earlier (or, word 15 of
      // rank 0's group, by rank 0 itself before it comes here)
      while ((v = peek(p)) == EMPTY) __builtin_amdgcn_s_sleep(1);
      words[k][lane] = v;
    }
  }
  // (A barrier later:) the value carried into this chunk; the last chunk of a group passes its
  // result on.
  __device__ __forceinline__ float carry(const Words<W> &words, const Map &m) const {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane >= W) return 0.f;
    float y = __uint_as_float((unsigned)words[GROUP - 1][lane]);
    for (int i = 0; i < j; ++i) {
      const unsigned long long v = words[i][lane];
      y = apply(__uint_as_float((unsigned)(v >> 32)), __uint_as_float((unsigned)v), y);
    }
    if (wave == 0 && j == GROUP - 1 && rank + 1 < NC)
      publish(pre + (size_t)(grp + 1) * W, word(0.f, apply(m.A, m.H, y)));
    return y;
  }
};

// ---- Forward -----------------------------------------------------------------
// A thread keeps its steps' decays and inputs in fp32 for the replay (64 registers for bf16;
// computing them again made that kernel bound by the vector unit).
template <typename T, bool MIX, bool PACKED> __global__ __launch_bounds__(THR, 4) void scan_fwd(ScanArgs a) {
  constexpr int C = CPT<T>, W = TC<T>;
  __shared__ __align__(16) Maps<W> s;
  __shared__ Words<W> words;
  const Offsets offs(a);
  const Place p = place<T>(a);
  const int tid = threadIdx.x, grp = tid / LPR, cl = (tid % LPR) * C, ch = p.c0 + cl;
  const int t0 = p.rank * CHUNK + grp * SEG;
  const int end = PACKED ? min(offs.last(), a.T) : a.T;
  const Steps<T, SEG> st(a, p.row, p.rank, grp, end, ch);
  u4 xr[SEG], gr[SEG];
  st.load(a.x, xr);
  st.load(a.g, gr);
  Marks m{0, 0};
  if (PACKED) {
    m = marks_of<SEG>(offs, t0, end);
    if (ch >= a.D) m = Marks{0, 0};
    copy_empty<C>(a, a.init, a.final_state, p.rank, grp, GRPS, ch);
  }
  st.mask(xr);
  st.mask(gr);

  // this thread's map; h0 keeps the initial state of the last sequence that starts here (another
  // workgroup may write its final state, which may be the same memory, before the replay below)
  float A[C], H[C], h0[C] = {}, lam[SEG][C], u[SEG][C];
#pragma unroll
  for (int c = 0; c < C; ++c) { A[c] = 1.f; H[c] = 0.f; }
#pragma unroll
  for (int i = 0; i < SEG; ++i) {
    if (PACKED && ((m.first >> i) & 1)) {
      load_seq<C>(a, a.init, t0 + i, ch, h0);
#pragma unroll
      for (int c = 0; c < C; ++c) { A[c] = -0.f; H[c] = h0[c]; }
    }
    step_of<MIX, C>(xr[i], gr[i], lam[i], u[i]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      A[c] *= lam[i][c];
      H[c] = fmaf(lam[i][c], H[c], u[i][c]);
    }
  }
  store_f32<C>(&s.A[grp][cl], A);
  store_f32<C>(&s.H[grp][cl], H);
  const float *first = !PACKED && a.init && p.c0 + (tid & 63) < a.D ? a.init + (size_t)p.row * a.D + p.c0 : nullptr;
  wave_map<W, false>(s);
  // a lone chunk: every wave reads it before the barrier, as wave 0 may write its memory after
  float y = a.NC == 1 && first && (tid & 63) < W ? first[tid & 63] : 0.f;
  __syncthreads();
  const Map m0 = chunk_map<W, false>(s);
  if (a.NC > 1) {
    const Chain<W> chain(a, p.col, p.rank);
    chain.give(m0, first);
    chain.take(words);
    __syncthreads();
    y = chain.carry(words, m0);
  }
  spread<W, false>(s, y);
  const float out = apply(m0.A, m0.H, y);
  if (tid < W && p.c0 + tid < a.D) {
    if (a.states) a.states[((size_t)p.row * a.NC + p.rank) * a.D + p.c0 + tid] = out;
    if (!PACKED && a.final_state && p.rank == a.NC - 1) a.final_state[(size_t)p.row * a.D + p.c0 + tid] = out;
  }
  float h[C];
  load_f32<C>(&s.H[grp][cl], h);
#pragma unroll
  for (int i = 0; i < SEG; ++i) {
    if (PACKED && ((m.first >> i) & 1)) {
      if (m.first >> (i + 1)) {   // a sequence inside these steps: read again, this thread alone writes its end
        load_seq<C>(a, a.init, t0 + i, ch, h);
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) h[c] = h0[c];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) h[c] = fmaf(lam[i][c], h[c], u[i][c]);
    st.store(a.h, i, pack16(h));
    if (PACKED && ((m.last >> i) & 1)) store_seq<C>(a, a.final_state, t0 + i, ch, h);
  }
}

// ---- Backward ----------------------------------------------------------------
// The states of the forward's chunks give the state entering a chunk, so only the reverse
// direction is chained (rank 0 is the last chunk).
// KEEP: the last steps whose 1 - lam is kept from the forward replay to the reverse one, as many as
// registers hold: bf16, 4 x 4096 x 768: none 37.6 us, 1 37.2, 2 37.0, 3 36.1, 4 (6 spilled) 39.2.
// Packed, where 6 registers are spilled with 1 and 8 with 3: 45.6 us each (16384 x 768, 13 sequences).
template <typename T, bool MIX, bool PACKED> __global__ __launch_bounds__(THR, 4) void scan_bwd(ScanArgs a) {
  constexpr int C = CPT<T>, W = TC<T>, KEEP = sizeof(T) == 4 ? SEG : PACKED ? 1 : 3;
  __shared__ __align__(16) union { Maps<W> s; Words<W> words; } f;   // forward maps; done with, the chain's words
  __shared__ __align__(16) Maps<W> s;                                 // reverse maps
  const Offsets offs(a);
  const Place p = place<T>(a);
  const int chunk = a.NC - 1 - p.rank;
  const int tid = threadIdx.x, grp = tid / LPR, cl = (tid % LPR) * C, ch = p.c0 + cl;
  const int t0 = chunk * CHUNK + grp * SEG;
  const int end = PACKED ? min(offs.last(), a.T) : a.T;
  const Steps<T, SEG> st(a, p.row, chunk, grp, end, ch);
  u4 xr[SEG], gr[SEG], dr[SEG];
  st.load(a.dh, dr);
  st.load(a.g, gr);
  st.load(a.x, xr);
  Marks m{0, 0};
  if (PACKED) {
    m = marks_of<SEG>(offs, t0, end);
    if (ch >= a.D) m = Marks{0, 0};
    copy_empty<C>(a, a.d_final, a.d_init, p.rank, grp, GRPS, ch);
  }
  st.mask(dr);
  st.mask(gr);

  // The reverse map of these steps first, r_{t+1} of the last to r_t of the first: others wait
  // for this chunk's, while the forward direction needs nobody.
  float A[C], H[C], lam[SEG][C];
#pragma unroll
  for (int c = 0; c < C; ++c) { A[c] = 1.f; H[c] = 0.f; }
#pragma unroll
  for (int i = SEG - 1; i >= 0; --i) {
    if (PACKED && ((m.last >> i) & 1)) {
      load_seq<C>(a, a.d_final, t0 + i, ch, H);
#pragma unroll
      for (int c = 0; c < C; ++c) A[c] = -0.f;
    }
    float gv[C], dv[C];
    unpack16(gr[i], gv);
    unpack16(dr[i], dv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lam[i][c] = decay(gv[c]);
      A[c] *= lam[i][c];
      H[c] = lam[i][c] * (dv[c] + H[c]);
    }
  }
  store_f32<C>(&s.A[grp][cl], A);
  store_f32<C>(&s.H[grp][cl], H);
  wave_map<W, true>(s);
  if (MIX) forget(gr);
  forget(dr);
  st.mask(xr);
#pragma unroll
  for (int c = 0; c < C; ++c) { A[c] = 1.f; H[c] = 0.f; }
#pragma unroll
  for (int i = 0; i < SEG; ++i) {
    if (PACKED && ((m.first >> i) & 1)) {
      load_seq<C>(a, a.init, t0 + i, ch, H);
#pragma unroll
      for (int c = 0; c < C; ++c) A[c] = -0.f;
    }
    float gv[C], u[C];
    unpack16(gr[i], gv);
    unpack16(xr[i], u);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (MIX) u[c] *= one_minus_decay(gv[c], lam[i][c]);
      A[c] *= lam[i][c];
      H[c] = fmaf(lam[i][c], H[c], u[c]);
    }
  }
  store_f32<C>(&f.s.A[grp][cl], A);
  store_f32<C>(&f.s.H[grp][cl], H);
  wave_map<W, false>(f.s);
  const bool on = p.c0 + (tid & 63) < a.D;
  const size_t c0 = (size_t)p.row * a.D + p.c0;
  const float *last = on && !PACKED && a.d_final ? a.d_final + c0 : nullptr;
  __syncthreads();
  const Map mr = chunk_map<W, true>(s);
  const Chain<W> chain(a, p.col, p.rank);
  if (a.NC > 1) chain.give(mr, last);
  float y = 0.f;
  if (on && (tid & 63) < W) {
    if (chunk > 0) y = a.states[((size_t)p.row * a.NC + chunk - 1) * a.D + p.c0 + (tid & 63)];
    else if (!PACKED && a.init) y = a.init[c0 + (tid & 63)];
  }
  spread<W, false>(f.s, y);
  forget(xr);
  forget(gr);
  float h[C], e[SEG][C], w[KEEP][C];      // e: what dlam multiplies, h_{t-1} (mix: h_{t-1} - x_t); w (mix): 1 - lam
  load_f32<C>(&f.s.H[grp][cl], h);
#pragma unroll
  for (int i = 0; i < SEG; ++i) {
    if (PACKED && ((m.first >> i) & 1)) load_seq<C>(a, a.init, t0 + i, ch, h);
    float gv[C], xv[C];
    unpack16(gr[i], gv);
    unpack16(xr[i], xv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]), omd = MIX ? one_minus_decay(gv[c], lam) : 1.f;
      if (MIX && i >= SEG - KEEP) w[i - (SEG - KEEP)][c] = omd;
      e[i][c] = MIX ? h[c] - xv[c] : h[c];
      h[c] = fmaf(lam, h[c], MIX ? omd * xv[c] : xv[c]);
    }
    // formed here and now: left to itself, the compiler keeps what they are made of instead
#pragma unroll
    for (int c = 0; c < C; ++c) {
      asm volatile("" : "+v"(e[i][c]), "+v"(h[c]));
      if (MIX && i >= SEG - KEEP) asm volatile("" : "+v"(w[i - (SEG - KEEP)][c]));
    }
  }
  y = 0.f;
  if (a.NC > 1) {
    __syncthreads();                      // every wave is done with the forward maps, whose place the words take
    chain.take(f.words);
    __syncthreads();
    y = chain.carry(f.words, mr);
  } else if (last && (tid & 63) < W) {
    y = last[tid & 63];
  }
  spread<W, true>(s, y);
  if (tid < W && on && !PACKED && a.d_init && chunk == 0) a.d_init[c0 + tid] = apply(mr.A, mr.H, y);
  forget(gr);
  forget(dr);
  float r[C];
  load_f32<C>(&s.H[grp][cl], r);
#pragma unroll
  for (int i = SEG - 1; i >= 0; --i) {
    if (PACKED && ((m.last >> i) & 1)) load_seq<C>(a, a.d_final, t0 + i, ch, r);
    float gv[C], dv[C], ox[C], og[C];
    unpack16(gr[i], gv);
    unpack16(dr[i], dv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lam = decay(gv[c]);
      const float delta = dv[c] + r[c];
      r[c] = lam * delta;
      ox[c] = MIX ? (i >= SEG - KEEP ? w[i - (SEG - KEEP)][c] : one_minus_decay(gv[c], lam)) * delta : delta;
      og[c] = r[c] * e[i][c];
    }
    st.store(a.dx, i, pack16(ox));
    st.store(a.dg, i, pack16(og));
    if (PACKED && ((m.first >> i) & 1)) store_seq<C>(a, a.d_init, t0 + i, ch, r);
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
  unpack16(*reinterpret_cast<const u4 *>(x + i), xv);
  unpack16(*reinterpret_cast<const u4 *>(g + i), gv);
  load_f32<C>(state + i, s);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float lam = decay(gv[c]);
    s[c] = fmaf(lam, s[c], MIX ? one_minus_decay(gv[c], lam) * xv[c] : xv[c]);
  }
  store_f32<C>(state + i, s);
  *reinterpret_cast<u4 *>(h + i) = pack16(s);
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

int64_t blocks_of(bool bf16, int rows, int T, int D) {
  const int tc = bf16 ? TC<__bf16> : TC<float>;
  return (int64_t)rows * ((D + tc - 1) / tc) * (((int64_t)T + CHUNK - 1) / CHUNK);
}

// Lays the workspace out, fills it, and gives the grid size.
hipError_t prepare(bool bf16, ScanArgs &a, void *ws, unsigned &grid, hipStream_t s) {
  a.NC = (a.T + CHUNK - 1) / CHUNK;
  grid = (unsigned)blocks_of(bf16, a.rows, a.T, a.D);
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

bool scan_fits(bool bf16, int rows, int T, int D) { return grid_fits(blocks_of(bf16, rows, T, D), THR); }

size_t scan_workspace(bool bf16, int rows, int T, int D) {
  const Layout l = layout(bf16, rows, T, D);
  return l.ticket + l.agg + l.pre;
}

#define FALCON_SCAN_LAUNCH(KERNEL)                                                                              \
  unsigned grid = 0;                                                                                            \
  const hipError_t e = prepare(bf16, a, ws, grid, s);                                                           \
  if (e != hipSuccess) return e;                                                                                \
  switch ((bf16 ? 4 : 0) + (mix ? 2 : 0) + (a.cu ? 1 : 0)) {                                                    \
    case 0: hipLaunchKernelGGL((KERNEL<float, false, false>), dim3(grid), dim3(THR), 0, s, a); break;           \
    case 1: hipLaunchKernelGGL((KERNEL<float, false, true>), dim3(grid), dim3(THR), 0, s, a); break;            \
    case 2: hipLaunchKernelGGL((KERNEL<float, true, false>), dim3(grid), dim3(THR), 0, s, a); break;            \
    case 3: hipLaunchKernelGGL((KERNEL<float, true, true>), dim3(grid), dim3(THR), 0, s, a); break;             \
    case 4: hipLaunchKernelGGL((KERNEL<__bf16, false, false>), dim3(grid), dim3(THR), 0, s, a); break;          \
    case 5: hipLaunchKernelGGL((KERNEL<__bf16, false, true>), dim3(grid), dim3(THR), 0, s, a); break;           \
    case 6: hipLaunchKernelGGL((KERNEL<__bf16, true, false>), dim3(grid), dim3(THR), 0, s, a); break;           \
    default: hipLaunchKernelGGL((KERNEL<__bf16, true, true>), dim3(grid), dim3(THR), 0, s, a);                  \
  }                                                                                                             \
  return hipGetLastError();

hipError_t launch_scan_fwd(bool bf16, bool mix, ScanArgs a, void *ws, hipStream_t s) {
  FALCON_SCAN_LAUNCH(scan_fwd)
}
hipError_t launch_scan_bwd(bool bf16, bool mix, ScanArgs a, void *ws, hipStream_t s) {
  FALCON_SCAN_LAUNCH(scan_bwd)
}
#undef FALCON_SCAN_LAUNCH

hipError_t launch_scan_step(bool bf16, bool mix, const void *x, const void *g, float *state, void *h, size_t n,
                            hipStream_t s) {
  const size_t blocks = (n / (bf16 ? 8 : 4) + 255) / 256;
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
