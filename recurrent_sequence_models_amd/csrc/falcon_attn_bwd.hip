// Causal softmax attention with grouped heads over packed sequences, backward, on gfx950.
//
// With P = e^{s - lse} (recomputed), D_i = do_i . o_i:
//   dv_j = sum_i P_ij do_i,  dS_ij = P_ij (do_i . v_j - D_i),
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i  (over the group's heads).
// Three kernels: the row sums D; one over key tiles for dk and dv; one over row tiles for
// dq.  The scores and do . v are formed twice (7 products of the size of the scores where
// 5 would do), and in return every sum is one wave's own, in a fixed order: no atomics, no
// fp32 copy of dq in memory, and equal inputs give equal bits.
//
// Rows are (token, head of the group) pairs as in the forward pass.  In the key kernel a
// wave owns 32 keys with their k and v in registers and forms S = Q K^T, so that P and dS
// are right operands of dV^T = dO^T P and dK^T = Q^T dS; in the row kernel a wave owns 32
// rows and forms the transposes.
//
// Bound: MFMA, 14 d flops executed per visible pair and head (10 d needed).
#include "attn_frag.h"
#include "layer_kernels.h"
#include "lane_ops.h"

namespace falcon {
namespace {

constexpr int THR = 256, TR = 128;   // 4 waves of 32 rows (or keys)

template <typename T, int D> __global__ __launch_bounds__(THR) void attn_delta(AttnArgs a, size_t nrow) {
  constexpr int E = 16 / (int)sizeof(T), L = D / E;
  const size_t row = ((size_t)blockIdx.x * THR + threadIdx.x) / L;
  const int e = (threadIdx.x % L) * E;
  float s = 0.f;
  if (row < nrow) {
    const size_t tok = row / a.hq, hq = row - tok * a.hq;
    const T *o = static_cast<const T *>(a.o) + tok * a.ldo + hq * D + e;
    const T *g = static_cast<const T *>(a.d_o) + tok * a.lddo + hq * D + e;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf((float)o[i], (float)g[i], s);
  }
  s = lane_sum<(L < 16 ? L : 16)>(s);
  if constexpr (L == 32) s = add_xor16(s);
  if (row < nrow && e == 0) a.delta[row] = s;
}

// ---- dk, dv ------------------------------------------------------------------
template <typename T, int D>
__global__ __launch_bounds__(THR, sizeof(T) * D > 256 ? 1 : 2) void attn_bwd_kv(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TQ = 32, DB = D / 16, CB = D / 32;
  typedef Copy<T, D, TQ> Cp;
  __shared__ uint4 sq[2][Cp::CH], sg[2][Cp::CH];
  __shared__ __align__(16) float sL[2][TQ], sD[2][TQ];   // lse (base 2) and D of the rows
  __shared__ __align__(16) int sM[2][TQ];                // the last key each row sees
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % (unsigned)a.hk, slot = blockIdx.x / (unsigned)a.hk;
  int n, tile;
  if (a.cuk) {
    const Slot s = find_slot(a.cuk, a.n, slot, 1, TR);
    n = s.n; tile = s.tile;
  } else {
    n = slot % (unsigned)a.n; tile = slot / (unsigned)a.n;
  }
  const Seq q = seq_of(a, n);
  if (tile >= (q.Lk + TR - 1) / TR) return;               // tile 0, which most rows see, starts first
  const int key0 = tile * TR, wkey = key0 + wave * 32, key = wkey + c;
  const bool on = key < q.Lk;
  const int rows = q.Lq * a.group, off = q.Lk - q.Lq;
  // the first row that sees a key of this tile, down to a whole tile of rows
  const int r_first = min(max(key0 - off, 0), q.Lq) * a.group / TQ * TQ;
  const int tiles = (rows - r_first + TQ - 1) / TQ;

  Frag<T> kf[DB], vf[DB];
  {
    const T *kp = static_cast<const T *>(a.k) + (int64_t)(q.k0 + min(key, q.Lk - 1)) * a.ldk + head * D;
    const T *vp = static_cast<const T *>(a.v) + (int64_t)(q.k0 + min(key, q.Lk - 1)) * a.ldv + head * D;
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      kf[b] = global_frag(kp, b, h);
      vf[b] = global_frag(vp, b, h);
    }
  }
  // Copying tiles of rows: rows past the sequence's repeat its last one, and their weights are
  // 0 (lse = inf).  A row's token is its number over the group, by a multiplication: exact for
  // the numbers up to group + 31 left when the tile's first token is taken off.
  const T *qg = static_cast<const T *>(a.q) + (int64_t)q.q0 * a.ldq + head * a.group * D;
  const T *gg = static_cast<const T *>(a.d_o) + (int64_t)q.q0 * a.lddo + head * a.group * D;
  const float inv = 1.f / a.group;
  auto token = [&](int rel) { return (int)((rel + 0.5f) * inv); };
  float rl = 0.f, rd = 0.f;
  int rm = 0;
  auto copy = [&](int t, int buf) {
    const int rt = r_first + t * TQ, tb = rt / (unsigned)a.group, r0 = tb * a.group;
    const T *qp = qg + (int64_t)tb * a.ldq, *gp = gg + (int64_t)tb * a.lddo;
#pragma unroll
    for (int i = 0; i < Cp::PER; ++i) {
      if (!Cp::has(i, wave)) continue;
      const int rel = min(rt + Cp::row(i, tid), rows - 1) - r0, tok = token(rel), hh = rel - tok * a.group;
      const unsigned in = hh * D * sizeof(T) + Cp::byte(i, tid);
      copy_to_lds(qp, tok * (unsigned)a.ldq * sizeof(T) + in, Cp::to(sq[buf], i, wave));
      copy_to_lds(gp, tok * (unsigned)a.lddo * sizeof(T) + in, Cp::to(sg[buf], i, wave));
    }
    if (tid < TQ) {
      rl = INFINITY; rd = 0.f; rm = -1;
      if (rt + tid < rows) {
        const int rel = rt + tid - r0, tok = token(rel), hh = rel - tok * a.group;
        const int64_t at = (int64_t)(q.q0 + tb + tok) * a.hq + head * a.group + hh;
        const float lse = a.lse_in[at];
        rl = lse == -INFINITY ? INFINITY : lse * kLog2e;   // a row that sees nothing
        rd = a.delta[at];
        rm = tb + tok + off;
      }
    }
  };
  auto hand_over = [&](int buf) {
    if (tid < TQ) { sL[buf][tid] = rl; sD[buf][tid] = rd; sM[buf][tid] = rm; }
    copies_done();
    __syncthreads();
  };
  f16v dk[CB], dv[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) dk[b] = dv[b] = zero16();
  const float sc = a.scale * kLog2e;
  if (tiles > 0) copy(0, 0);
  hand_over(0);
  for (int t = 0; t < tiles; ++t) {
    const int buf = t & 1, rt = r_first + t * TQ;
    if (t + 1 < tiles) copy(t + 1, buf ^ 1);               // its last readers are behind the barrier
    const int first_lim = (int)(rt / (unsigned)a.group) + off;
    const int last_lim = (int)(min(rt + TQ - 1, rows - 1) / (unsigned)a.group) + off;
    if (wkey <= last_lim) {                                // else no row of the tile sees a key of this wave
      f16v s = zero16(), g = zero16();
#pragma unroll
      for (int b = 0; b < DB; ++b) mma(s, Ti::rows(sq[buf], 0, b, lane), kf[b]);
#pragma unroll
      for (int b = 0; b < DB; ++b) mma(g, Ti::rows(sg[buf], 0, b, lane), vf[b]);
      const bool masked = wkey + 31 > first_lim;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f4 L = *reinterpret_cast<const f4 *>(&sL[buf][8 * b + 4 * h]);
        const f4 Dr = *reinterpret_cast<const f4 *>(&sD[buf][8 * b + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * b + i] = __builtin_amdgcn_exp2f(fmaf(s[4 * b + i], sc, -L[i]));
        if (masked) {
          const int4 M = *reinterpret_cast<const int4 *>(&sM[buf][8 * b + 4 * h]);
          const int lim[4] = {M.x, M.y, M.z, M.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) s[4 * b + i] = key > lim[i] ? 0.f : s[4 * b + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) g[4 * b + i] = s[4 * b + i] * (g[4 * b + i] - Dr[i]);
      }
#pragma unroll
      for (int b16 = 0; b16 < 2; ++b16) {
        const Frag<T> pf = result_frag<T>(s, b16), gf = result_frag<T>(g, b16);
#pragma unroll
        for (int b = 0; b < CB; ++b) mma(dv[b], Ti::cols(sg[buf], b16 * 16, b * 32, lane), pf);
#pragma unroll
        for (int b = 0; b < CB; ++b) mma(dk[b], Ti::cols(sq[buf], b16 * 16, b * 32, lane), gf);
      }
    }
    hand_over(buf ^ 1);
  }
  if (!on) return;
  T *pk = static_cast<T *>(a.dk) + (int64_t)(q.k0 + key) * a.lddk + head * D;
  T *pv = static_cast<T *>(a.dv) + (int64_t)(q.k0 + key) * a.lddv + head * D;
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int e = b * 32 + 2 * i + 4 * h;
      store4(pk + e, dk[b][i] * a.scale, dk[b][i + 1] * a.scale, dk[b][i + 2] * a.scale, dk[b][i + 3] * a.scale);
      store4(pv + e, dv[b][i], dv[b][i + 1], dv[b][i + 2], dv[b][i + 3]);
    }
}

// ---- dq ----------------------------------------------------------------------
template <typename T, int D>
__global__ __launch_bounds__(THR, sizeof(T) * D > 256 ? 1 : 2) void attn_bwd_q(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TN = 32, DB = D / 16, CB = D / 32;
  typedef Copy<T, D, TN> Cp;
  __shared__ uint4 sk[2][Cp::CH], sv[2][Cp::CH];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % (unsigned)a.hk, slot = blockIdx.x / (unsigned)a.hk;
  int n, tile;
  if (a.cuq) {
    const Slot s = find_slot(a.cuq, a.n, slot, a.group, TR);
    n = s.n; tile = s.tile;
  } else {
    n = slot % (unsigned)a.n; tile = slot / (unsigned)a.n;
  }
  const Seq q = seq_of(a, n);
  const int rows = q.Lq * a.group, tiles = (rows + TR - 1) / TR;
  if (tile >= tiles) return;
  tile = tiles - 1 - tile;
  const int off = q.Lk - q.Lq, r0 = tile * TR + wave * 32, r = min(r0 + c, rows - 1);
  const bool on = r0 + c < rows;
  const int tok = r / (unsigned)a.group, hq = head * a.group + (r - tok * a.group);
  const int lim = tok + off;
  const int first_lim = (int)((unsigned)min(r0, rows - 1) / (unsigned)a.group) + off;
  const int wave_lim = (int)((unsigned)min(r0 + 31, rows - 1) / (unsigned)a.group) + off;
  const int last_lim = (int)((unsigned)min(tile * TR + TR - 1, rows - 1) / (unsigned)a.group) + off;
  const int keys = max(min(q.Lk, last_lim + 1), 0), ktiles = (keys + TN - 1) / TN;

  const T *qp = static_cast<const T *>(a.q) + (int64_t)(q.q0 + tok) * a.ldq + hq * D;
  const T *gp = static_cast<const T *>(a.d_o) + (int64_t)(q.q0 + tok) * a.lddo + hq * D;
  Frag<T> qf[DB], gf[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) { qf[b] = global_frag(qp, b, h); gf[b] = global_frag(gp, b, h); }
  const int64_t at = (int64_t)(q.q0 + tok) * a.hq + hq;
  float L = a.lse_in[at];
  L = L == -INFINITY ? INFINITY : L * kLog2e;
  const float Dr = a.delta[at];

  const T *kg = static_cast<const T *>(a.k) + (int64_t)q.k0 * a.ldk + head * D;
  const T *vg = static_cast<const T *>(a.v) + (int64_t)q.k0 * a.ldv + head * D;
  const unsigned kstep = (unsigned)a.ldk * sizeof(T), vstep = (unsigned)a.ldv * sizeof(T);
  auto copy = [&](int kt, int buf) {            // rows past the sequence's keys repeat its last one
    const T *kp = kg + (int64_t)kt * TN * a.ldk, *vp = vg + (int64_t)kt * TN * a.ldv;
    const int last = q.Lk - 1 - kt * TN;
#pragma unroll
    for (int i = 0; i < Cp::PER; ++i) {
      if (!Cp::has(i, wave)) continue;
      const int row = min(Cp::row(i, tid), last);
      copy_to_lds(kp, row * kstep + Cp::byte(i, tid), Cp::to(sk[buf], i, wave));
      copy_to_lds(vp, row * vstep + Cp::byte(i, tid), Cp::to(sv[buf], i, wave));
    }
  };
  f16v dq[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) dq[b] = zero16();
  const float sc = a.scale * kLog2e;
  if (ktiles > 0) copy(0, 0);
  copies_done();
  __syncthreads();
  for (int kt = 0; kt < ktiles; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < ktiles) copy(kt + 1, buf ^ 1);            // its last readers are behind the barrier
    if (kt * TN <= wave_lim) {
      f16v s = zero16(), g = zero16();
#pragma unroll
      for (int b = 0; b < DB; ++b) mma(s, Ti::rows(sk[buf], 0, b, lane), qf[b]);
#pragma unroll
      for (int b = 0; b < DB; ++b) mma(g, Ti::rows(sv[buf], 0, b, lane), gf[b]);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], sc, -L));
      if (kt * TN + TN - 1 > first_lim) {
        const int left = lim - kt * TN - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + (i & 3) > left ? 0.f : s[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] *= g[i] - Dr;
#pragma unroll
      for (int b16 = 0; b16 < 2; ++b16) {
        const Frag<T> sf = result_frag<T>(s, b16);
#pragma unroll
        for (int b = 0; b < CB; ++b) mma(dq[b], Ti::cols(sk[buf], b16 * 16, b * 32, lane), sf);
      }
    }
    copies_done();
    __syncthreads();
  }
  if (!on) return;
  T *pq = static_cast<T *>(a.dq) + (int64_t)(q.q0 + tok) * a.lddq + hq * D;
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      store4(pq + b * 32 + 2 * i + 4 * h, dq[b][i] * a.scale, dq[b][i + 1] * a.scale, dq[b][i + 2] * a.scale,
             dq[b][i + 3] * a.scale);
}

int64_t query_rows(const AttnArgs &a) { return a.cuq ? (int64_t)a.Tq : (int64_t)a.n * a.Tq; }

template <typename T, int D> hipError_t run(AttnArgs &a, hipStream_t s) {
  const size_t nrow = (size_t)query_rows(a) * a.hq;
  constexpr int L = D * (int)sizeof(T) / 16;
  const int64_t kslots = a.cuk ? (int64_t)a.Tk / TR + a.n : ((int64_t)a.Tk + TR - 1) / TR * a.n;
  const int64_t qslots = a.cuq ? (int64_t)a.Tq * a.group / TR + a.n : ((int64_t)a.Tq * a.group + TR - 1) / TR * a.n;
  const size_t nb = (nrow * L + THR - 1) / THR;
  if (nb > 0x7fffffff || kslots * a.hk > 0x7fffffff || qslots * a.hk > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((attn_delta<T, D>), dim3((unsigned)nb), dim3(THR), 0, s, a, nrow);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_bwd_kv<T, D>), dim3((unsigned)(kslots * a.hk)), dim3(THR), 0, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((attn_bwd_q<T, D>), dim3((unsigned)(qslots * a.hk)), dim3(THR), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t attn_bwd_workspace(const AttnArgs &a) { return (size_t)query_rows(a) * a.hq * sizeof(float); }

hipError_t launch_attn_bwd(bool bf16, int d, AttnArgs a, void *ws, hipStream_t s) {
  a.delta = static_cast<float *>(ws);
#define FALCON_ATTN(D_) \
  if (d == D_) return bf16 ? run<__bf16, D_>(a, s) : run<float, D_>(a, s)
  FALCON_ATTN(32);
  FALCON_ATTN(64);
  FALCON_ATTN(128);
#undef FALCON_ATTN
  return hipErrorInvalidValue;
}

}  // namespace falcon
