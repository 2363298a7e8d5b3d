// Causal softmax attention with grouped heads over packed sequences, backward, on gfx950.
//
// With P = e^{s - lse} (recomputed), D_i = do_i . o_i:
//   dv_j = sum_i P_ij do_i,  dS_ij = P_ij (do_i . v_j - D_i),
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i  (over the group's heads).
// Two kernels: one over row tiles for D and dq, one over key tiles for dk and dv.  The scores
// and do . v are formed twice (7 products of the size of the scores where 5 would do), and in
// return every sum is one wave's own, in a fixed order: no atomics, no fp32 copy of dq in
// memory, and equal inputs give equal bits.
//
// Roundings, for bf16: P and dS as operands of the products that sum over them (8-bit mantissas are
// what the matrix unit takes at this rate; each adds 0.16 % of a gradient's norm to the 0.17 % of its
// own rounding: 0.23 to 0.25 % in all).  D is fp32, although o is rounded, in dk and in the dq of rows
// that see 128 keys at most (with D from the rounded o: 0.79 % at 2 tokens, 0.27 % at 64).  Over more
// keys dq takes it from o, which adds less than 0.02 % where a row's weight is spread; where it lies on
// few of 2048 keys (scores of standard deviation 2.5) dq is off by 0.41 %: one more product over all
// keys, a tenth of the time, would be the price of the rest.  Sums are fp32.
//
// Rows are (token, head of the group) pairs as in the forward pass.  In the key kernel a
// wave owns 32 keys with their k and v in registers and forms S = Q K^T, so that P and dS
// are right operands of dV^T = dO^T P and dK^T = Q^T dS; in the row kernel a wave owns 32
// rows and forms the transposes.
//
// Bound: the matrix unit, 14 d flops executed per visible pair and head (10 d needed), and power
// (operands of zeros: 20 % less time).  Measured, as useful flops (10 d), where an 8192^3 bf16
// matrix product reaches 1.21 PFLOP/s:
//   4 x 4096, 16 / 4 heads of 128, bf16: 0.98 ms, 700 TFLOP/s (in a long run 1.11: rows 399 us, keys
//     687, their sum 27)
//   8 x 2048, 12 / 12 heads of 64, bf16: 213 us, 605 TFLOP/s (in a long run 260: rows 115 us, keys 144)
//   2 x 2048, 12 / 12 heads of 64, fp32: 526 us, 61 TFLOP/s
#include "attn_frag.h"
#include "layer_kernels.h"
#include "lane_ops.h"

namespace falcon {
namespace {

constexpr int THR = 256, TR = 128;   // 4 waves of 32 rows (or keys)

// ---- dq ----------------------------------------------------------------------
// Three waves a SIMD where rows are 128 bytes at most (167 registers at bf16, d = 64).
template <typename T, int D>
__global__ __launch_bounds__(THR, sizeof(T) * D > 256 ? 1 : sizeof(T) * D > 128 ? 2 : 3) void attn_bwd_q(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TN = 64, DB = D / 16, CB = D / 32;   // keys of a tile (32: 1 to 2 % more time)
  typedef Copy<T, D, TN> Cp;
  __shared__ uint4 sk[2][Cp::CH], sv[2][Cp::CH];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, c = lane & 31, h = lane >> 5;
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
  if ((unsigned)tile >= (unsigned)tiles) return;
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
  // -D = -do . o, where the products do . v start from, and lse in base 2, +inf where the row sees
  // nothing, so that all its weights e^{s - lse} come out 0.
  // o is rounded, and what D is off by is the same in all do . v - D of a row: for bf16 the largest
  // error there is in rows whose weight lies on few keys.  As the weights add up to 1, the sum over
  // the keys of P (do . v - D) is what D lacks.  It is summed beside the products, so that the key
  // kernel gets a D of fp32 throughout; rows that see two tiles of keys at most, which both stand in
  // LDS, form it first, so that dq has it as well.  Forward and backward of 8 x 2048, 12 / 12 heads of
  // 64, in a long run: 281 us without the sum, 287 with it; of 16 x 128 the same 30 us.
  constexpr bool SUMS = sizeof(T) == 2;
  const int64_t at = (int64_t)(q.q0 + tok) * a.hq + hq;
  const T *op = static_cast<const T *>(a.o) + at * D;
  float Dr = 0.f;
#pragma unroll
  for (int b = 0; b < DB; ++b) Dr -= dot(global_frag(op, b, h), gf[b]);
  Dr = add_xor32(Dr);
  const float lse = a.lse_in[at], L = lse == -INFINITY ? INFINITY : lse * kLog2e;
  if (on && h == 0) a.lse2[at] = L;             // for the key kernel, as -D below

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
  const float sc = a.scale * kLog2e;
  // P, and do . v - D, of the 32 keys from key0 (kb of the tile in buf)
  auto products = [&](int buf, int kb, int key0, f16v &s, f16v &g) {
    s = zero16();
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = Dr;
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(s, Ti::rows(sk[buf], kb, b, lane), qf[b]);
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(g, Ti::rows(sv[buf], kb, b, lane), gf[b]);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], sc, -L));
    if (key0 + 31 > first_lim) {
      const int left = lim - key0 - 4 * h;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + (i & 3) > left ? 0.f : s[i];
    }
  };
  const bool refine = SUMS && ktiles <= 2;
  if (ktiles > 0) copy(0, 0);
  if (refine && ktiles == 2) copy(1, 1);
  copies_done();
#pragma unroll
  for (int b = 0; b < DB; ++b) { arrived(qf[b]); arrived(gf[b]); }
  __syncthreads();
  float rest = 0.f;                             // the sum over the keys of P (do . v - D), 0 but for D's error
  if (refine) {
    for (int key0 = 0; key0 < ktiles * TN && key0 <= wave_lim; key0 += 32) {
      f16v s, g;
      products(key0 / TN, key0 % TN, key0, s, g);
#pragma unroll
      for (int i = 0; i < 16; ++i) rest = fmaf(s[i], g[i], rest);
    }
    Dr -= add_xor32(rest);
    rest = 0.f;
  }
  f16v dq[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) dq[b] = zero16();
  for (int kt = 0; kt < ktiles; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < ktiles && !refine) copy(kt + 1, buf ^ 1);  // its last readers are behind the barrier
#pragma unroll
    for (int kb = 0; kb < TN; kb += 32) {
      const int key0 = kt * TN + kb;
      if (key0 > wave_lim) break;               // no row of this wave sees the keys from here on
      f16v s, g;
      products(buf, kb, key0, s, g);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] *= g[i];
      if (SUMS)
#pragma unroll
        for (int i = 0; i < 16; ++i) rest += s[i];
#pragma unroll
      for (int b16 = 0; b16 < 2; ++b16) {
        const Frag<T> sf = result_frag<T>(s, b16);
#pragma unroll
        for (int b = 0; b < CB; ++b) mma(dq[b], Ti::cols(sk[buf], kb + b16 * 16, b * 32, lane), sf);
      }
    }
    copies_done();
    __syncthreads();
  }
  if (SUMS) Dr -= add_xor32(rest);
  if (!on) return;
  if (h == 0) a.delta[at] = Dr;                 // for the key kernel
  T *pq = static_cast<T *>(a.dq) + (int64_t)(q.q0 + tok) * a.lddq + hq * D;
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      store4(pq + b * 32 + 2 * i + 4 * h, dq[b][i] * a.scale, dq[b][i + 1] * a.scale, dq[b][i + 2] * a.scale,
             dq[b][i + 3] * a.scale);
}

// ---- dk, dv ------------------------------------------------------------------
// Rows of a tile: 64 (half the barriers and address work of 32: 8 x 2048, 12 heads of 64, bf16,
// 228 us for the whole backward against 237), or 32 where two pairs of tiles of 64 would leave one
// workgroup a compute unit.
template <typename T, int D> constexpr int TQ_OF = sizeof(T) * D > 128 ? 32 : 64;
// Where rows are longer than 128 bytes, the values wait in LDS instead of registers, and at bf16,
// d = 128, 2 of a lane's 8 key fragments: with both operands and both sums in registers (192 of
// the 256 that leave two waves a SIMD) the compiler spills, and every reload waits for the copies
// in flight as well.  4 x 4096, 16 / 4 heads of 128: 0.96 ms, with the keys in registers 1.05, with
// the values too 1.46; fp32 rows of 64, which fit either way, the same.  Two workgroups' LDS still fit.
template <typename T, int D> constexpr bool V_IN_LDS = sizeof(T) * D > 128;
template <typename T, int D> constexpr int KEYS_IN_LDS = sizeof(T) == 2 && D == 128 ? 2 : 0;

template <typename T, int D>
__global__ __launch_bounds__(THR, sizeof(T) * D > 256 ? 1 : 2) void attn_bwd_kv(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TQ = TQ_OF<T, D>, DB = D / 16, CB = D / 32;
  constexpr bool VL = V_IN_LDS<T, D>;
  typedef Copy<T, D, TQ> Cp;
  typedef Copy<T, D, TR> CpV;
  constexpr int KR = DB - KEYS_IN_LDS<T, D>;
  __shared__ uint4 sq[2][Cp::CH], sg[2][Cp::CH], sv[VL ? CpV::CH : 1];
  __shared__ Frag<T> sk[DB > KR ? DB - KR : 1][THR];
  __shared__ __align__(16) float sL[2][64], sD[2][64];   // lse (base 2) and -D of the rows
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, c = lane & 31, h = lane >> 5;
  unsigned id = blockIdx.x;
  const int head = id % (unsigned)a.hk;
  id /= (unsigned)a.hk;
  const int split = id % (unsigned)a.splits, slot = id / (unsigned)a.splits;
  int n, tile;
  if (a.cuk) {
    const Slot s = find_slot(a.cuk, a.n, slot, 1, TR);
    n = s.n; tile = s.tile;
  } else {
    n = slot % (unsigned)a.n; tile = slot / (unsigned)a.n;
  }
  const Seq q = seq_of(a, n);
  if ((unsigned)tile >= (unsigned)((q.Lk + TR - 1) / TR)) return;   // tile 0, which most rows see, starts first
  const int key0 = tile * TR, wkey = key0 + wave * 32, key = wkey + c;
  const bool on = key < q.Lk;
  const int rows = q.Lq * a.group, off = q.Lk - q.Lq;
  // The first row that sees a key: of this lane's, of any of this wave's, of all of them, and,
  // down to a whole tile of rows, of any of this tile's; then this split's share of the tiles.
  auto first_row = [&](int k) { return max(min(k, q.Lk - 1) - off, 0) * a.group; };
  const int see = first_row(key), wave_see = first_row(wkey), wave_all = first_row(wkey + 31);
  const int r_first = first_row(key0) / TQ * TQ;
  const int64_t all = (rows - r_first + TQ - 1) / TQ;
  const int t0 = __builtin_amdgcn_readfirstlane((int)(all * split / a.splits));
  const int t1 = __builtin_amdgcn_readfirstlane((int)(all * (split + 1) / a.splits));

  Frag<T> kf[KR], vf[VL ? 1 : DB];
  {
    const T *kp = static_cast<const T *>(a.k) + (int64_t)(q.k0 + min(key, q.Lk - 1)) * a.ldk + head * D;
    const T *vp = static_cast<const T *>(a.v) + (int64_t)(q.k0 + min(key, q.Lk - 1)) * a.ldv + head * D;
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      if (b < KR) kf[b < KR ? b : 0] = global_frag(kp, b, h);
      else sk[b < KR ? 0 : b - KR][tid] = global_frag(kp, b, h);
      if (!VL) vf[VL ? 0 : b] = global_frag(vp, b, h);
    }
  }
  if (VL) {
    const T *vg = static_cast<const T *>(a.v) + (int64_t)(q.k0 + key0) * a.ldv + head * D;
#pragma unroll
    for (int i = 0; i < CpV::PER; ++i) {
      const int row = min(CpV::row(i, tid), q.Lk - 1 - key0);
      copy_to_lds(vg, row * (unsigned)a.ldv * sizeof(T) + CpV::byte(i, tid), CpV::to(sv, i, wave));
    }
  }
  auto keys = [&](int b) { return b < KR ? kf[b < KR ? b : 0] : sk[b < KR ? 0 : b - KR][tid]; };
  auto value = [&](int b) { return VL ? Ti::rows(sv, wave * 32, b, lane) : vf[VL ? 0 : b]; };
  // Copying tiles of rows: rows past the sequence's repeat its last one, and their weights are
  // masked.  A row's token is its number over the group, by a multiplication: in 64 bits it is
  // exact for any row number, in 32 for the numbers up to group + 63 left when the tile's first
  // token is taken off.
  const T *qg = static_cast<const T *>(a.q) + (int64_t)q.q0 * a.ldq + head * a.group * D;
  const T *gg = static_cast<const T *>(a.d_o) + (int64_t)q.q0 * a.lddo + head * a.group * D;
  const int64_t row0 = (int64_t)q.q0 * a.hq + head * a.group;
  const double inv64 = 1.0 / a.group;
  const float inv = (float)inv64;
  auto token64 = [&](int row) { return __builtin_amdgcn_readfirstlane((int)((row + 0.5) * inv64)); };
  auto token = [&](int rel) { return (int)((rel + 0.5f) * inv); };
  auto copy = [&](int t, int buf) {
    const int rt = r_first + t * TQ, tb = token64(rt), r0 = tb * a.group;
    const T *qp = qg + (int64_t)tb * a.ldq, *gp = gg + (int64_t)tb * a.lddo;
#pragma unroll
    for (int i = 0; i < Cp::PER; ++i) {
      if (!Cp::has(i, wave)) continue;
      const int rel = min(rt + Cp::row(i, tid), rows - 1) - r0, tok = token(rel), hh = rel - tok * a.group;
      const unsigned in = hh * D * sizeof(T) + Cp::byte(i, tid);
      copy_to_lds(qp, tok * (unsigned)a.ldq * sizeof(T) + in, Cp::to(sq[buf], i, wave));
      copy_to_lds(gp, tok * (unsigned)a.lddo * sizeof(T) + in, Cp::to(sg[buf], i, wave));
    }
    if (wave < 2) {
      const int rel = min(rt + lane, rows - 1) - r0, tok = token(rel), hh = rel - tok * a.group;
      const int64_t at = row0 + (int64_t)tb * a.hq;
      copy4_to_lds((wave ? a.delta : a.lse2) + at, (tok * (unsigned)a.hq + hh) * 4,
                   lds_address(wave ? sD[buf] : sL[buf]));
    }
  };
  f16v dk[CB], dv[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) dk[b] = dv[b] = zero16();
  const float sc = a.scale * kLog2e;
  if (t0 < t1) copy(t0, 0);
  copies_done();
#pragma unroll
  for (int b = 0; b < KR; ++b) arrived(kf[b]);
#pragma unroll
  for (int b = 0; b < (VL ? 0 : DB); ++b) arrived(vf[b]);
  __syncthreads();
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    if (t + 1 < t1) copy(t + 1, buf ^ 1);                  // its last readers are behind the barrier
    // what the tile's first and last rows see
    const int rt = r_first + t * TQ;
    const int lo = see - rt - 4 * h, hi = rows - rt - 4 * h;   // the rows of the tile that see this lane's key
    const bool masked = rt < wave_all || rt + TQ > rows;
    if (rt + TQ > wave_see)                                // else no row of the tile sees a key of this wave
#pragma unroll
    for (int rb = 0; rb < TQ; rb += 32) {
      if (rt + rb >= rows) break;
      f16v s = zero16(), g;
#pragma unroll
      for (int b = 0; b < DB; ++b) mma(s, Ti::rows(sq[buf], rb, b, lane), keys(b));
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f4 Dr = *reinterpret_cast<const f4 *>(&sD[buf][rb + 8 * b + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[4 * b + i] = Dr[i];
      }
#pragma unroll
      for (int b = 0; b < DB; ++b) mma(g, Ti::rows(sg[buf], rb, b, lane), value(b));
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f4 L = *reinterpret_cast<const f4 *>(&sL[buf][rb + 8 * b + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * b + i] = __builtin_amdgcn_exp2f(fmaf(s[4 * b + i], sc, -L[i]));
      }
      if (masked) {   // the same for the whole wave; once, so that what is around it stays in two pieces
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = rb + 8 * (i / 4) + (i & 3);
          s[i] = e >= lo && e < hi ? s[i] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] *= s[i];
#pragma unroll
      for (int b16 = 0; b16 < 2; ++b16) {
        const Frag<T> pf = result_frag<T>(s, b16), gf = result_frag<T>(g, b16);
#pragma unroll
        for (int b = 0; b < CB; ++b) mma(dv[b], Ti::cols(sg[buf], rb + b16 * 16, b * 32, lane), pf);
#pragma unroll
        for (int b = 0; b < CB; ++b) mma(dk[b], Ti::cols(sq[buf], rb + b16 * 16, b * 32, lane), gf);
      }
    }
    copies_done();
    __syncthreads();
  }
  if (!on) return;
  if (a.splits > 1) {   // [split][dk, dv][key token, head][d]
    const size_t nkey = (size_t)key_tokens(a) * a.hk, at = (size_t)(q.k0 + key) * a.hk + head;
    float *pk = a.part + ((size_t)split * 2 * nkey + at) * D, *pv = pk + nkey * D;
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = b * 32 + 2 * i + 4 * h;
        store4(pk + e, dk[b][i], dk[b][i + 1], dk[b][i + 2], dk[b][i + 3]);
        store4(pv + e, dv[b][i], dv[b][i + 1], dv[b][i + 2], dv[b][i + 3]);
      }
    return;
  }
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

// Adds the splits of dk and dv in order: one thread per 4 entries.
template <typename T, int D> __global__ __launch_bounds__(THR) void attn_bwd_sum(AttnArgs a, size_t nkey) {
  constexpr int L = D / 4;
  const size_t at = ((size_t)blockIdx.x * THR + threadIdx.x) / L;
  const int e = (threadIdx.x % L) * 4;
  if (at >= nkey) return;
  const size_t tok = at / a.hk;
  const int head = (int)(at - tok * a.hk);
  if (a.cuk && tok >= (size_t)max(a.cuk[a.n], 0)) return;      // behind the last sequence
  f4 dk = zero4(), dv = zero4();
  for (int s = 0; s < a.splits; ++s) {
    const float *p = a.part + ((size_t)s * 2 * nkey + at) * D + e;
    dk += *reinterpret_cast<const f4 *>(p);
    dv += *reinterpret_cast<const f4 *>(p + nkey * D);
  }
  dk *= a.scale;
  store4(static_cast<T *>(a.dk) + (int64_t)tok * a.lddk + head * D + e, dk[0], dk[1], dk[2], dk[3]);
  store4(static_cast<T *>(a.dv) + (int64_t)tok * a.lddv + head * D + e, dv[0], dv[1], dv[2], dv[3]);
}

int64_t key_slots(const AttnArgs &a) {
  return a.cuk ? (int64_t)a.Tk / TR + a.n : ((int64_t)a.Tk + TR - 1) / TR * a.n;
}
int64_t row_slots(const AttnArgs &a) {
  return a.cuq ? (int64_t)a.Tq * a.group / TR + a.n : ((int64_t)a.Tq * a.group + TR - 1) / TR * a.n;
}
int64_t sum_blocks(const AttnArgs &a, int d) { return (key_tokens(a) * a.hk * (d / 4) + THR - 1) / THR; }

// Splits of the rows between workgroups of one key tile.  Tile 0 meets every row and the last
// tile 128 of them, so at two workgroups a compute unit one round of workgroups would take
// twice the average one; with 1024 of them the short ones fill in.  At least 512 rows (of the
// average sequence) a split, so that writing and adding the parts stays small beside them.
// 1 x 4096, 16 / 4 heads of 128: 0.30 ms, unsplit 0.83, for 512 workgroups 0.34, for 2048 0.34;
// 4 x 4096: 0.96, 1.14, 1.14, 0.99; 8 x 2048, 12 / 12 heads of 64, is not split: 228 us, 293 in two.
int bwd_splits(const AttnArgs &a) {
  const int64_t blocks = key_slots(a) * a.hk;
  const int64_t rows = (a.cuq ? a.Tq / a.n : a.Tq) * (int64_t)a.group;
  int64_t s = (1024 + blocks - 1) / blocks;
  if (s > rows / 512) s = rows / 512;
  if (s > 16) s = 16;
  return s < 1 ? 1 : (int)s;
}

template <typename T, int D> hipError_t run(AttnArgs &a, hipStream_t s) {
  const size_t nkey = (size_t)key_tokens(a) * a.hk;
  const unsigned nk = (unsigned)(key_slots(a) * a.hk * a.splits), nq = (unsigned)(row_slots(a) * a.hk);
  hipLaunchKernelGGL((attn_bwd_q<T, D>), dim3(nq), dim3(THR), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_bwd_kv<T, D>), dim3(nk), dim3(THR), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((attn_bwd_sum<T, D>), dim3((unsigned)sum_blocks(a, D)), dim3(THR), 0, s, a, nkey);
  return hipGetLastError();
}

// One fp32 number per query and head, in whole 16 bytes.
size_t row_bytes(const AttnArgs &a) { return ((size_t)query_tokens(a) * a.hq * sizeof(float) + 15) & ~(size_t)15; }

}  // namespace

bool attn_bwd_fits(int d, const AttnArgs &a) {
  const int splits = bwd_splits(a);
  return grid_fits(row_slots(a) * a.hk, THR) && grid_fits(key_slots(a) * a.hk * splits, THR) &&
         (splits == 1 || grid_fits(sum_blocks(a, d), THR));
}

size_t attn_bwd_workspace(int d, const AttnArgs &a) {
  const int s = bwd_splits(a);
  const size_t part = s == 1 ? 0 : (size_t)s * 2 * key_tokens(a) * a.hk * d * sizeof(float);
  return 2 * row_bytes(a) + part;
}

hipError_t launch_attn_bwd(bool bf16, int d, AttnArgs a, void *ws, hipStream_t s) {
  unsigned char *p = static_cast<unsigned char *>(ws);
  a.splits = bwd_splits(a);
  a.delta = reinterpret_cast<float *>(p);
  a.lse2 = reinterpret_cast<float *>(p + row_bytes(a));
  a.part = reinterpret_cast<float *>(p + 2 * row_bytes(a));
#define FALCON_ATTN(D_) \
  if (d == D_) return bf16 ? run<__bf16, D_>(a, s) : run<float, D_>(a, s)
  FALCON_ATTN(32);
  FALCON_ATTN(64);
  FALCON_ATTN(128);
#undef FALCON_ATTN
  return hipErrorInvalidValue;
}

}  // namespace falcon
