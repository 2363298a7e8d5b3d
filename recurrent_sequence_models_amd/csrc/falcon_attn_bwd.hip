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

struct Seq { int q0, Lq, k0, Lk; };
__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int n) {
  if (a.cuq) return Seq{a.cuq[n], a.cuq[n + 1] - a.cuq[n], a.cuk[n], a.cuk[n + 1] - a.cuk[n]};
  return Seq{n * a.Tq, a.Tq, n * a.Tk, a.Tk};
}

// ---- dk, dv ------------------------------------------------------------------
template <typename T, int D> __global__ __launch_bounds__(THR, 1) void attn_bwd_kv(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TQ = 32, CH = TQ * Ti::CPR, PER = (CH + THR - 1) / THR, DB = D / 16, CB = D / 32;
  __shared__ uint4 sq[2][CH], sg[2][CH];
  __shared__ __align__(16) float sL[2][TQ], sD[2][TQ];   // lse (base 2) and D of the rows
  __shared__ __align__(16) int sM[2][TQ];                // the last key each row sees
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % a.hk, slot = blockIdx.x / a.hk;
  int n, tile;
  if (a.cuk) {
    const Slot s = find_slot(a.cuk, a.n, slot, 1, TR);
    n = s.n; tile = s.tile;
  } else {
    n = slot % a.n; tile = slot / a.n;
  }
  const Seq q = seq_of(a, n);
  if (tile >= (q.Lk + TR - 1) / TR) return;               // tile 0, which most rows see, starts first
  const int key0 = tile * TR, key = key0 + wave * 32 + c;
  const bool on = key < q.Lk;
  const int64_t rows = (int64_t)q.Lq * a.group;
  const int off = q.Lk - q.Lq;
  // the first row that sees a key of this tile, down to a whole tile of rows
  const int64_t r_first = min((int64_t)max(key0 - off, 0) * a.group, rows) / TQ * TQ;
  const int tiles = (int)((rows - r_first + TQ - 1) / TQ);

  Frag<T> kf[DB], vf[DB];
  {
    const T *kp = static_cast<const T *>(a.k) + (int64_t)(q.k0 + key) * a.ldk + head * D;
    const T *vp = static_cast<const T *>(a.v) + (int64_t)(q.k0 + key) * a.ldv + head * D;
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      kf[b] = vf[b] = zero_frag(T());
      if (on) { kf[b] = global_frag(kp, b, h); vf[b] = global_frag(vp, b, h); }
    }
  }
  uint4 qr[PER], gr[PER];
  float rl = 0.f, rd = 0.f;
  int rm = 0;
  auto fetch = [&](int t) {
    const int64_t rt = r_first + (int64_t)t * TQ;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * THR, row = e / Ti::CPR, ch = e % Ti::CPR;
      const int64_t r = rt + row;
      qr[i] = gr[i] = uint4{0, 0, 0, 0};
      if (e < CH && r < rows) {
        const int tok = (int)(r / a.group), hq = head * a.group + (int)(r - (int64_t)tok * a.group);
        qr[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + (int64_t)(q.q0 + tok) * a.ldq + hq * D + ch * Ti::E);
        gr[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.d_o) + (int64_t)(q.q0 + tok) * a.lddo + hq * D + ch * Ti::E);
      }
    }
    if (tid < TQ) {
      const int64_t r = rt + tid;
      rl = INFINITY; rd = 0.f; rm = -1;                    // rows outside: P = e^-inf = 0
      if (r < rows) {
        const int tok = (int)(r / a.group), hq = head * a.group + (int)(r - (int64_t)tok * a.group);
        const int64_t at = (int64_t)(q.q0 + tok) * a.hq + hq;
        const float lse = a.lse_in[at];
        rl = lse == -INFINITY ? INFINITY : lse * kLog2e;   // a row that sees nothing
        rd = a.delta[at];
        rm = tok + off;
      }
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * THR, row = e / Ti::CPR, ch = e % Ti::CPR;
      if (e < CH) {
        sq[buf][Ti::place(row, ch)] = qr[i];
        sg[buf][Ti::place(row, ch)] = gr[i];
      }
    }
    if (tid < TQ) { sL[buf][tid] = rl; sD[buf][tid] = rd; sM[buf][tid] = rm; }
  };
  f16v dk[CB], dv[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) dk[b] = dv[b] = zero16();
  const float sc = a.scale * kLog2e;
  if (tiles > 0) { fetch(0); stage(0); }
  __syncthreads();
  for (int t = 0; t < tiles; ++t) {
    const int buf = t & 1;
    if (t + 1 < tiles) fetch(t + 1);
    f16v s = zero16(), g = zero16();
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(s, Ti::rows(sq[buf], 0, b, lane), kf[b]);
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(g, Ti::rows(sg[buf], 0, b, lane), vf[b]);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f4 L = *reinterpret_cast<const f4 *>(&sL[buf][8 * b + 4 * h]);
      const f4 Dr = *reinterpret_cast<const f4 *>(&sD[buf][8 * b + 4 * h]);
      const int4 M = *reinterpret_cast<const int4 *>(&sM[buf][8 * b + 4 * h]);
      const int lim[4] = {M.x, M.y, M.z, M.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p = __builtin_amdgcn_exp2f(fmaf(s[4 * b + i], sc, -L[i]));
        if (key > lim[i]) p = 0.f;
        s[4 * b + i] = p;
        g[4 * b + i] = p * (g[4 * b + i] - Dr[i]);
      }
    }
#pragma unroll
    for (int b16 = 0; b16 < 2; ++b16) {
      const Frag<T> pf = result_frag<T>(s, b16), gf = result_frag<T>(g, b16);
#pragma unroll
      for (int b = 0; b < CB; ++b) mma(dv[b], Ti::cols(sg[buf], b16 * 16, b * 32, lane), pf);
#pragma unroll
      for (int b = 0; b < CB; ++b) mma(dk[b], Ti::cols(sq[buf], b16 * 16, b * 32, lane), gf);
    }
    if (t + 1 < tiles) stage(buf ^ 1);
    __syncthreads();
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
template <typename T, int D> __global__ __launch_bounds__(THR, 1) void attn_bwd_q(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TN = 32, CH = TN * Ti::CPR, PER = (CH + THR - 1) / THR, DB = D / 16, CB = D / 32;
  __shared__ uint4 sk[2][CH], sv[2][CH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % a.hk, slot = blockIdx.x / a.hk;
  int n, tile;
  if (a.cuq) {
    const Slot s = find_slot(a.cuq, a.n, slot, a.group, TR);
    n = s.n; tile = s.tile;
  } else {
    n = slot % a.n; tile = slot / a.n;
  }
  const Seq q = seq_of(a, n);
  const int64_t rows = (int64_t)q.Lq * a.group;
  const int tiles = (int)((rows + TR - 1) / TR);
  if (tile >= tiles) return;
  tile = tiles - 1 - tile;
  const int off = q.Lk - q.Lq;
  const int64_t r = (int64_t)tile * TR + wave * 32 + c;
  const bool on = r < rows;
  const int tok = (int)((on ? r : rows - 1) / a.group), hq = head * a.group + (int)((on ? r : rows - 1) % a.group);
  const int lim = tok + off;
  const int last_lim = (int)(min((int64_t)tile * TR + TR - 1, rows - 1) / a.group) + off;
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
  uint4 kr[PER], vr[PER];
  auto fetch = [&](int kt) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * THR, row = e / Ti::CPR, ch = e % Ti::CPR;
      const int key = kt * TN + row;
      kr[i] = vr[i] = uint4{0, 0, 0, 0};
      if (e < CH && key < q.Lk) {
        kr[i] = *reinterpret_cast<const uint4 *>(kg + (int64_t)key * a.ldk + ch * Ti::E);
        vr[i] = *reinterpret_cast<const uint4 *>(vg + (int64_t)key * a.ldv + ch * Ti::E);
      }
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * THR, row = e / Ti::CPR, ch = e % Ti::CPR;
      if (e < CH) {
        sk[buf][Ti::place(row, ch)] = kr[i];
        sv[buf][Ti::place(row, ch)] = vr[i];
      }
    }
  };
  f16v dq[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) dq[b] = zero16();
  const float sc = a.scale * kLog2e;
  if (ktiles > 0) { fetch(0); stage(0); }
  __syncthreads();
  for (int kt = 0; kt < ktiles; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < ktiles) fetch(kt + 1);
    f16v s = zero16(), g = zero16();
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(s, Ti::rows(sk[buf], 0, b, lane), qf[b]);
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(g, Ti::rows(sv[buf], 0, b, lane), gf[b]);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = kt * TN + 8 * (i / 4) + 4 * h + (i & 3);
      float p = __builtin_amdgcn_exp2f(fmaf(s[i], sc, -L));
      if (key > lim) p = 0.f;
      s[i] = p * (g[i] - Dr);
    }
#pragma unroll
    for (int b16 = 0; b16 < 2; ++b16) {
      const Frag<T> sf = result_frag<T>(s, b16);
#pragma unroll
      for (int b = 0; b < CB; ++b) mma(dq[b], Ti::cols(sk[buf], b16 * 16, b * 32, lane), sf);
    }
    if (kt + 1 < ktiles) stage(buf ^ 1);
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
