// Selective state-space scan on gfx950, backward.
//
// With gy_t = dy_t silu(z_t), a_t = exp(delta_t A), against time:
//   g_t = gy_t C_t + r_{t+1},  r_t = a_t g_t           (r behind the last step: d_final)
//   dC_t = sum_d gy_t h_t,  dB_t = sum_d g_t delta_t x_t
//   dx_t = delta_t sum_n g_t B_t + D gy_t
//   ddelta_t = sum_n (r_t h_{t-1} A + g_t B_t x_t),  ddt_t = ddelta_t softplus'
//   dA = sum_t r_t h_{t-1} delta_t,  dD = sum_t gy_t x_t,  dbias = sum_t ddt_t
//   dz_t = dy_t (sum_n C_t h_t + D x_t) silu'(z_t),  d init = r at the first step.
//
// The layout of the forward, its tiles taken from the last to the first.  A tile starts from the state
// that the forward kept; its waves compose their 16 steps in both directions (the maps share their
// factor exp(A sum of delta)), join the maps, run forward again to have the states before their steps in
// registers beside the decays, and then back.  Sums over the states are over 4 registers and N / 4
// lanes; those over the channels, for dB and dC, go by exchanges that halve the number of values with the
// number of lanes (16 instructions for 8 sums over 16 lanes), over the waves in LDS, and over
// workgroups in a pass of their own, in order.
//
// Bound: the vector unit: 112 instructions for 4 states and a step (62 in the way back, 32 in the maps of both
// directions and the run forward, 18 for what a tile's loading, gates and results cost), 79 % busy.  A lane's decays and
// states of 16 steps take 132 registers, so a SIMD has two waves.  Measured, N = 16, bf16: 4 x 4096 x 1536 430 us and 45 for
// the maps (192 sequences' workgroups on 256 compute units; 545 with whole sequences), and 18 us for dB and dC over the 48
// groups of channels.
#include "ssm_common.h"

namespace falcon {
namespace {

// v_permlane16_swap / v_permlane32_swap of the pairs (a0, b0), (a1, b1), then their sums: rows (halves) of
// even number get the sum of two rows of a, odd ones that of b.  Every lane of the wave calls it.
__device__ __forceinline__ void halve16(float a0, float b0, float a1, float b1, float &x0, float &x1) {
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\tv_permlane16_swap_b32 %2, %3\n\ts_nop 1"
               : "+v"(a0), "+v"(b0), "+v"(a1), "+v"(b1));
  x0 = a0 + b0;
  x1 = a1 + b1;
}
__device__ __forceinline__ void halve32(float a0, float b0, float a1, float b1, float &x0, float &x1) {
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\tv_permlane32_swap_b32 %2, %3\n\ts_nop 1"
               : "+v"(a0), "+v"(b0), "+v"(a1), "+v"(b1));
  x0 = a0 + b0;
  x1 = a1 + b1;
}
// Sums over the channels of a wave: u = b[r], v = c[r] of row r = lane / 16, in each lane of its part of the states.
template <int P> __device__ __forceinline__ void channel_sums(const f4 &b, const f4 &c, float &u, float &v) {
  float q0, q1, q2, q3;
  halve16(b[0], b[1], b[2], b[3], q0, q1);
  halve16(c[0], c[1], c[2], c[3], q2, q3);
  halve32(q0, q1, q2, q3, u, v);
  if constexpr (P <= 4) { u += dpp_mov<0x124>(u); v += dpp_mov<0x124>(v); }    // row_ror:4
  if constexpr (P <= 8) { u += dpp_mov<0x128>(u); v += dpp_mov<0x128>(v); }    // row_ror:8
}

template <int N> using BwdTile = SsmTile<N, SSM_BWD_CH, 64 / N, 16>;
// Workgroups begin in the order of their numbers: the sequences' first segments, which are never the shorter ones, come first.
__device__ __forceinline__ int bwd_slot(const SeqMap &q, int len, int i) {
  return q.cu ? i : i % q.n * segments_of(q, len) + i / q.n;
}

// MAPS: only the segment's map (r at its start from zero behind its end, sum of delta) is formed.
template <typename T, int N, bool MAPS> __global__ __launch_bounds__(BwdTile<N>::THR, MAPS ? 4 : 2) void ssm_bwd(SsmArgs a) {
  typedef BwdTile<N> L;
  static_assert(L::TS == SSM_CHUNK<N>, "a tile starts from a state that the forward kept");
  constexpr int V = L::VEC, BV = L::BV, CH = SSM_BWD_CH;
  __shared__ __align__(16) f4 step[L::TS][CH];               // (delta, delta x, gy, -); then (sum g B, sum r h A log2 e, sum C h, -)
  __shared__ __align__(16) float sBC[L::TS][2][N];
  __shared__ __align__(16) float map[L::TW][3][CH][N];       // P, G and H of the waves' steps
  __shared__ __align__(16) float red[MAPS ? 1 : L::WIDE][L::TS][2 * N];
  __shared__ float sumd[L::TW][CH], sbias[CH], sskip[CH];
  const int groups = (a.D + CH - 1) / CH;
  const SsmPlace place = ssm_place(groups, slots_of(a.seq, a.seg));
  if (!place.any) return;
  const Segment g = find_segment(a.seq, a.seg, bwd_slot(a.seq, a.seg, place.slot));
  const int group = place.group, c0 = group * CH;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tw = wave / L::WIDE, wide = wave % L::WIDE, p = lane % L::P, p4 = p * 4, ch = wide * L::CW + lane / L::P;
  const int c = c0 + ch;
  const bool on = c < a.D;
  const int ls = tid / (CH / V), lc = (tid % (CH / V)) * V, lcc = c0 + lc;
  const bool lon = lcc < a.D;
  const bool empty = g.s == g.e && g.slot == first_slot(a.seq, g.n, a.seg);
  const bool first = g.t0 == g.s, lastseg = g.t1 == g.e;
  if constexpr (MAPS) {
    if (!g.any || first) return;        // nobody starts from its end
  }
  f4 A2{0.f, 0.f, 0.f, 0.f}, r{0.f, 0.f, 0.f, 0.f};
  if (on) {
    A2 = *reinterpret_cast<const f4 *>(a.A + (size_t)c * N + p4) * SSM_LOG2E;
    if constexpr (!MAPS) {
      if (g.any && !lastseg) r = *reinterpret_cast<const f4 *>(a.seg_state + ((size_t)g.slot * a.D + c) * N + p4);
      else if ((g.any || empty) && a.d_final) r = *reinterpret_cast<const f4 *>(a.d_final + ((size_t)g.n * a.D + c) * N + p4);
    }
  }
  const int bs = tid / (N / BV), bn = (tid % (N / BV)) * BV;
  if (tid < CH) {
    sbias[tid] = a.bias && c0 + tid < a.D ? a.bias[c0 + tid] : 0.f;
    sskip[tid] = a.skip && c0 + tid < a.D ? a.skip[c0 + tid] : 0.f;
  }
  __syncthreads();
  const int chunk0 = MAPS ? 0 : first_slot(a.seq, g.n, L::TS);
  f4 dA{0.f, 0.f, 0.f, 0.f};
  float dD[V] = {}, dbias[V] = {}, total = 0.f;
  const int64_t tokens = a.seq.tokens();
  Few<T, V> nx{}, nd, nz, ng;                 // the next tile's entries of this thread
  Few<T, BV> nB, nC;
  f4 nh{0.f, 0.f, 0.f, 0.f};                  // and its first state
  auto load = [&](int t) {
    const int q = min(ls, g.t1 - 1 - t), qb = min(bs, g.t1 - 1 - t), cc = lon ? lcc : 0;
    if constexpr (!MAPS) fetch(entry<T>(a.x, a.ldx, t, q, cc), nx);
    fetch(entry<T>(a.dt, a.lddt, t, q, cc), nd);
    if (a.z) fetch(entry<T>(a.z, a.ldz, t, q, cc), nz);
    fetch(entry<T>(a.dy, a.D, t, q, cc), ng);
    if (!MAPS) fetch(entry<T>(a.B, a.ldB, t, qb, bn), nB);
    fetch(entry<T>(a.C, a.ldC, t, qb, bn), nC);
    if constexpr (!MAPS) {
      if (on) nh = *reinterpret_cast<const f4 *>(a.states + ((size_t)(chunk0 + (t - g.s) / L::TS) * a.D + c) * N + p4);
    }
  };
  const int last = g.any ? g.t0 + (g.t1 - g.t0 - 1) / L::TS * L::TS : g.t0 - 1;     // the last tile
  if (last >= g.t0) load(last);
  for (int t = last; t >= g.t0; t -= L::TS) {
    const bool valid = lon && t + ls < g.t1;     // steps behind the end change nothing: delta = gy = 0
    const Few<T, V> x = nx;
    float d[V], slope[V], gy[V], gz[V];          // gz: dz but for its factor sum C h + D x
    f4 hv = nh;                                  // the tile's first state, then this wave's
#pragma unroll
    for (int j = 0; j < V; ++j) {
      d[j] = nd[j] + sbias[lc + j];
      slope[j] = 1.f;
      if (a.softplus) { slope[j] = sigmoid(d[j]); d[j] = softplus(d[j]); }
      gy[j] = ng[j];
      if (a.z) {
        const float z = nz[j], sg = sigmoid(z);
        gz[j] = gy[j] * sg * fmaf(z, 1.f - sg, 1.f);
        gy[j] *= z * sg;
      }
      step[ls][lc + j] = valid ? f4{d[j], d[j] * x[j], gy[j], 0.f} : f4{0.f, 0.f, 0.f, 0.f};
    }
    const bool there = t + bs < g.t1;            // and B = C = 0: the last token's may be infinite
#pragma unroll
    for (int j = 0; j < BV; ++j) {
      if (!MAPS) sBC[bs][0][bn + j] = there ? nB[j] : 0.f;
      sBC[bs][1][bn + j] = there ? nC[j] : 0.f;
    }
    __syncthreads();
    if (t > g.t0) load(t - L::TS);
    const int s0 = tw * L::STEPS;
    f4 dec[L::STEPS];
    f4 mine = r;                                 // r behind this wave's steps
    if constexpr (L::TW > 1 || MAPS) {
      float sd = 0.f;
      f4 H{0.f, 0.f, 0.f, 0.f}, G{0.f, 0.f, 0.f, 0.f}, Pm;
#pragma unroll
      for (int s = 0; s < L::STEPS; ++s) {
        const f4 du = step[s0 + s][ch];
        sd += du[0];
#pragma unroll
        for (int j = 0; j < 4; ++j) dec[s][j] = __builtin_amdgcn_exp2f(du[0] * A2[j]);
        if constexpr (!MAPS) {
          const f4 b = *reinterpret_cast<const f4 *>(&sBC[s0 + s][0][p4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) H[j] = fmaf(dec[s][j], H[j], du[1] * b[j]);
        }
      }
#pragma unroll
      for (int s = L::STEPS - 1; s >= 0; --s) {
        const float gv = step[s0 + s][ch][2];
        const f4 cv = *reinterpret_cast<const f4 *>(&sBC[s0 + s][1][p4]);
#pragma unroll
        for (int j = 0; j < 4; ++j) G[j] = dec[s][j] * fmaf(gv, cv[j], G[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) Pm[j] = __builtin_amdgcn_exp2f(sd * A2[j]);
      *reinterpret_cast<f4 *>(&map[tw][0][ch][p4]) = Pm;
      *reinterpret_cast<f4 *>(&map[tw][1][ch][p4]) = G;
      if constexpr (!MAPS) *reinterpret_cast<f4 *>(&map[tw][2][ch][p4]) = H;
      if (MAPS && p4 == 0) sumd[tw][ch] = sd;
      __syncthreads();
      f4 run = r;
#pragma unroll
      for (int w = L::TW - 1; w >= 0; --w) {
        if (w == tw) mine = run;
        const f4 Pw = *reinterpret_cast<const f4 *>(&map[w][0][ch][p4]), Gw = *reinterpret_cast<const f4 *>(&map[w][1][ch][p4]);
#pragma unroll
        for (int j = 0; j < 4; ++j) run[j] = fmaf(Pw[j], run[j], Gw[j]);
        if (MAPS) total += sumd[w][ch];
      }
      r = run;
      if constexpr (!MAPS) {
#pragma unroll
        for (int w = 0; w < L::TW - 1; ++w) {
          if (w < tw) {
            const f4 Pw = *reinterpret_cast<const f4 *>(&map[w][0][ch][p4]), Hw = *reinterpret_cast<const f4 *>(&map[w][2][ch][p4]);
#pragma unroll
            for (int j = 0; j < 4; ++j) hv[j] = fmaf(Pw[j], hv[j], Hw[j]);
          }
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < L::STEPS; ++s) {
        const float delta = step[s0 + s][ch][0];
#pragma unroll
        for (int j = 0; j < 4; ++j) dec[s][j] = __builtin_amdgcn_exp2f(delta * A2[j]);
      }
    }
    if constexpr (!MAPS) {
      f4 hp[L::STEPS + 1];                       // the state before every step
      hp[0] = hv;
#pragma unroll
      for (int s = 0; s < L::STEPS; ++s) {
        const float du = step[s0 + s][ch][1];
        const f4 b = *reinterpret_cast<const f4 *>(&sBC[s0 + s][0][p4]);
#pragma unroll
        for (int j = 0; j < 4; ++j) hp[s + 1][j] = fmaf(dec[s][j], hp[s][j], du * b[j]);
      }
      // what comes now reads the tile again, rather than keep it in registers
      asm volatile("" ::: "memory");
      // the channels' 4 (of N = 32, 64: first 4) lanes store one sum each, and a row's first lanes of two channels those of
      // B and of C (the others the same values at the same places)
      float *out = reinterpret_cast<float *>(&step[s0][ch]) + (p & 3);
      const bool second = L::P < 16 && (lane / L::P) & 1;
      float *outr = &red[wide][s0][p4 + (lane >> 4) + (second ? N : 0)];
#pragma unroll
      for (int s = L::STEPS - 1; s >= 0; --s) {
        const f4 du = step[s0 + s][ch];
        const f4 b = *reinterpret_cast<const f4 *>(&sBC[s0 + s][0][p4]), cv = *reinterpret_cast<const f4 *>(&sBC[s0 + s][1][p4]);
        f4 gb, gc;
        float sum_b = 0.f, sum_a = 0.f, read = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gj = fmaf(du[2], cv[j], mine[j]);
          gb[j] = gj * du[1];
          gc[j] = du[2] * hp[s + 1][j];
          sum_b = fmaf(gj, b[j], sum_b);
          read = fmaf(cv[j], hp[s + 1][j], read);
          mine[j] = dec[s][j] * gj;
          const float w = mine[j] * hp[s][j];
          sum_a = fmaf(w, A2[j], sum_a);
          dA[j] = fmaf(w, du[0], dA[j]);
        }
        sum_b = lane_sum<L::P>(sum_b);
        sum_a = lane_sum<L::P>(sum_a);
        read = lane_sum<L::P>(read);
        float u, v;
        channel_sums<L::P>(gb, gc, u, v);
        if constexpr (L::P < 16) {
          outr[s * 2 * N] = second ? v : u;
        } else {
          outr[s * 2 * N] = u;
          outr[s * 2 * N + N] = v;
        }
        out[s * CH * 4] = (p & 3) == 0 ? sum_b : (p & 3) == 1 ? sum_a : read;
      }
      if constexpr (L::TW == 1) r = mine;
    }
    __syncthreads();
    if constexpr (!MAPS) {
      if (valid) {
        float dx[V], ddt[V], dz[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const f4 sum = step[ls][lc + j];
          const float xv = x[j], sk = sskip[lc + j];
          dx[j] = fmaf(sum[0], d[j], sk * gy[j]);
          ddt[j] = fmaf(sum[0], xv, sum[1] * SSM_LN2) * slope[j];
          dD[j] = fmaf(gy[j], xv, dD[j]);
          dbias[j] += ddt[j];
          if (a.z) dz[j] = gz[j] * fmaf(sk, xv, sum[2]);
        }
        put(entry<T>(a.dx, a.lddx, t, ls, lcc), dx);
        put(entry<T>(a.ddt, a.ldddt, t, ls, lcc), ddt);
        if (a.z) put(entry<T>(a.dz, a.lddz, t, ls, lcc), dz);
      }
      float *out = a.part_bc + ((size_t)group * tokens + t) * (2 * N);
#pragma unroll
      for (int k = 0; k < L::TS * 2 * N / 4 / L::THR; ++k) {
        const int i = (k * L::THR + tid) * 4;
        f4 v = *reinterpret_cast<const f4 *>(&red[0][0][0] + i);
#pragma unroll
        for (int w = 1; w < L::WIDE; ++w) v += *reinterpret_cast<const f4 *>(&red[w][0][0] + i);
        if (t + i / (2 * N) < g.t1) *reinterpret_cast<f4 *>(out + i) = v;
      }
    }
  }
  if constexpr (MAPS) {
    if (tw == 0 && on) {
      *reinterpret_cast<f4 *>(a.seg_map + ((size_t)g.slot * a.D + c) * N + p4) = r;
      if (p4 == 0) a.seg_sum[(size_t)g.slot * a.D + c] = total;
    }
  } else {
    if (tw == 0 && on && a.d_init && (empty || (g.any && first)))
      *reinterpret_cast<f4 *>(a.d_init + ((size_t)g.n * a.D + c) * N + p4) = r;
    // the segment's sums for A, D and the bias, over its waves (steps) in order; zeros without any
    __syncthreads();
    *reinterpret_cast<f4 *>(&map[tw][0][ch][p4]) = dA;
#pragma unroll
    for (int j = 0; j < V; ++j) step[ls][lc + j] = f4{dD[j], dbias[j], 0.f, 0.f};
    __syncthreads();
    if (on && tw == 0) {
#pragma unroll
      for (int w = 1; w < L::TW; ++w) dA += *reinterpret_cast<const f4 *>(&map[w][0][ch][p4]);
      *reinterpret_cast<f4 *>(a.part_A + ((size_t)g.slot * a.D + c) * N + p4) = dA;
    }
    if (tid < CH && c0 + tid < a.D) {
      float v = 0.f, w = 0.f;
      for (int i = 0; i < L::TS; ++i) {
        v += step[i][tid][0];
        w += step[i][tid][1];
      }
      float *out = a.part_D + (size_t)g.slot * 2 * a.D + c0 + tid;
      out[0] = v;
      out[a.D] = w;
    }
  }
}

// r behind every segment of a sequence but its last, in reverse order.
template <int N> __global__ __launch_bounds__(256) void ssm_chain_bwd(SsmArgs a) {
  const int per = a.D * (N / 4), i = blockIdx.x * 256 + threadIdx.x;
  if (i >= per) return;
  const int c = i / (N / 4), p4 = (i % (N / 4)) * 4;
  const f4 A2 = *reinterpret_cast<const f4 *>(a.A + (size_t)c * N + p4) * SSM_LOG2E;
  for (int n = blockIdx.y; n < a.seq.n; n += gridDim.y) {
    const int s = a.seq.begin(n), e = a.seq.end(n), slot = first_slot(a.seq, n, a.seg);
    f4 r{0.f, 0.f, 0.f, 0.f};
    if (a.d_final) r = *reinterpret_cast<const f4 *>(a.d_final + ((size_t)n * a.D + c) * N + p4);
    for (int k0 = e > s ? (e - s - 1) / a.seg : 0; k0 > 0; k0 -= CHAIN_AHEAD) {
      f4 G[CHAIN_AHEAD];
      float sd[CHAIN_AHEAD];
#pragma unroll
      for (int k = 0; k < CHAIN_AHEAD; ++k) {
        const size_t at = (size_t)(slot + max(k0 - k, 1)) * a.D + c;
        sd[k] = a.seg_sum[at];
        G[k] = *reinterpret_cast<const f4 *>(a.seg_map + at * N + p4);
      }
#pragma unroll
      for (int k = 0; k < CHAIN_AHEAD; ++k) {
        if (k0 - k <= 0) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = fmaf(__builtin_amdgcn_exp2f(sd[k] * A2[j]), r[j], G[k][j]);
        *reinterpret_cast<f4 *>(a.seg_state + ((size_t)(slot + k0 - k - 1) * a.D + c) * N + p4) = r;
      }
    }
  }
}

// dB and dC: the sums over the groups of channels, in order.
template <typename T, int N> __global__ __launch_bounds__(256) void ssm_sum_bc(SsmArgs a, int groups) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, tokens = a.seq.tokens();
  if (i >= tokens * 2 * N) return;
  const int64_t t = i / (2 * N);
  const int n = (int)(i % (2 * N));
  if (a.seq.cu && (t >= a.seq.end(a.seq.n - 1) || t < a.seq.begin(0))) return;      // tokens of no sequence
  f4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < groups; ++k) s += *reinterpret_cast<const f4 *>(a.part_bc + (size_t)k * tokens * (2 * N) + i);
  const float v[4] = {s[0], s[1], s[2], s[3]};
  if (n < N) put(static_cast<T *>(a.dB) + t * a.lddB + n, v);
  else put(static_cast<T *>(a.dC) + t * a.lddC + n - N, v);
}

struct Parts { size_t bc, A, D, map, sum, total; };
Parts parts_of(const SeqMap &q, int D, int N) {
  const int seg = ssm_segment_bwd(q, D, N);
  const size_t groups = (D + SSM_BWD_CH - 1) / SSM_BWD_CH, slots = slots_of(q, seg);
  Parts p;
  p.bc = align16(groups * q.tokens() * 2 * N * sizeof(float));
  p.A = align16(slots * D * N * sizeof(float));
  p.D = align16(slots * 2 * D * sizeof(float));
  const bool cut = ssm_segmented(q, seg);
  p.map = cut ? align16((slots + 1) * D * N * sizeof(float)) : 0;
  p.sum = cut ? align16((slots + 1) * D * sizeof(float)) : 0;
  p.total = p.bc + p.A + p.D + 2 * p.map + p.sum;
  return p;
}

}  // namespace

size_t ssm_bwd_workspace(SeqMap seq, int D, int N) { return parts_of(seq, D, N).total; }

template <typename T, int N> static hipError_t bwd(SsmArgs a, const SsmGrads &o, void *ws, hipStream_t s) {
  const Parts p = parts_of(a.seq, a.D, N);
  char *at = static_cast<char *>(ws);
  a.part_bc = reinterpret_cast<float *>(at);
  a.part_A = reinterpret_cast<float *>(at += p.bc);
  a.part_D = reinterpret_cast<float *>(at += p.A);
  a.seg_map = reinterpret_cast<float *>(at += p.D);
  a.seg_state = reinterpret_cast<float *>(at += p.map);
  a.seg_sum = reinterpret_cast<float *>(at += p.map);
  a.seg = ssm_segment_bwd(a.seq, a.D, N);
  const int groups = (a.D + SSM_BWD_CH - 1) / SSM_BWD_CH, slots = slots_of(a.seq, a.seg);
  const unsigned grid = (unsigned)ssm_grid(groups, slots);
  hipError_t e;
  if (ssm_segmented(a.seq, a.seg)) {
    hipLaunchKernelGGL((ssm_bwd<T, N, true>), dim3(grid), dim3(BwdTile<N>::THR), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int rows = a.seq.n < 65535 ? a.seq.n : 65535;
    hipLaunchKernelGGL((ssm_chain_bwd<N>), dim3((a.D * (N / 4) + 255) / 256, rows), dim3(256), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssm_bwd<T, N, false>), dim3(grid), dim3(BwdTile<N>::THR), 0, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t sums = (int64_t)a.seq.tokens() * 2 * N / 4;
  hipLaunchKernelGGL((ssm_sum_bc<T, N>), dim3((unsigned)((sums + 255) / 256)), dim3(256), 0, s, a, groups);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  e = launch_column_sum(a.part_A, slots, (int64_t)a.D * N, o.dA, (int64_t)a.D * N, nullptr, s);
  if (e != hipSuccess || (!o.dD && !o.dbias)) return e;
  return launch_column_sum(a.part_D, slots, 2 * (int64_t)a.D, o.dD, a.D, o.dbias, s);
}

hipError_t launch_ssm_bwd(bool bf16, int N, SsmArgs a, SsmGrads o, void *ws, hipStream_t s) {
  if (N == 16) return bf16 ? bwd<__bf16, 16>(a, o, ws, s) : bwd<float, 16>(a, o, ws, s);
  if (N == 32) return bf16 ? bwd<__bf16, 32>(a, o, ws, s) : bwd<float, 32>(a, o, ws, s);
  if (N == 64) return bf16 ? bwd<__bf16, 64>(a, o, ws, s) : bwd<float, 64>(a, o, ws, s);
  return hipErrorInvalidValue;
}

}  // namespace falcon
