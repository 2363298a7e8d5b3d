// Causal softmax attention with grouped heads over packed sequences, forward, on gfx950.
//
// Query i of a sequence sees keys j <= i + Lk - Lq (the queries are the last Lq of its Lk
// tokens).  Per query head, with s_ij = scale q_i . k_j:
//   o_i = sum_j e^{s_ij - m} v_j / l,  l = sum_j e^{s_ij - m},  lse_i = m + ln l,
// in one pass over the keys with the running maximum m and sum l; a query that sees no key
// gets o = 0 and lse = -inf.
//
// The rows of a tile are (token, head of the group) pairs, row r = token r / group, head
// r % group: the heads that share a key head share its tiles, and a single token still
// fills `group` rows.  A wave owns 32 rows and keeps their queries and results in
// registers; tiles of 64 keys and values pass through LDS.  Scores are formed transposed,
// S^T = K Q^T, so a lane holds 32 scores of one row: the softmax needs one exchange
// between two lanes, its factors need none, and P^T is the right operand of
// O^T = V^T P^T as it stands.
//
// Bound: for prompts the matrix unit (4 d flops per visible pair and head), with the
// exponentials close behind, and power: with operands of zeros the same launches take 20 %
// less, as the clock then stays up.  HBM (K and V once) for single tokens.  Measured, where an
// 8192^3 bf16 matrix product reaches 1.21 PFLOP/s:
//   1 x 16384, 16 / 4 heads of 128, bf16: 1.01 to 1.06 ms by the card, 1.04 to 1.09 PFLOP/s (matrix unit
//     busy 56 %, vector unit 54 %)
//   8 x 2048, 12 / 12 heads of 64, bf16: 76 us, 0.68 PFLOP/s (35 and 64 %), 92 us in a long run
//   2 x 2048, 12 / 12 heads of 64, fp32: 192 us, 67 TFLOP/s (384 workgroups; an fp32 product: 154)
// Issuing the next tile's scores between this one's exponentials, in one wave, was slower (80 us
// and 1.06 ms): the waves of a SIMD overlap the two by themselves, without its registers.
//
// Roundings, for bf16: the weights as operands of their product with v (8-bit mantissas are what the
// matrix unit takes at this rate), 0.16 % of the norm of o beside the 0.17 % of its own rounding: 0.19
// to 0.23 % in all.  Scores, the sum of weights and lse are fp32.
#include "attn_frag.h"
#include "layer_kernels.h"

namespace falcon {
namespace {

constexpr int THR = 256, TM = 128;   // 4 waves of 32 rows

template <typename T, int D> struct Fwd {
  // Keys of a tile: 64, or 32 where two pairs of tiles of 64 would take over 64 KB of LDS
  // (fp32 at d = 128).
  static constexpr int TN = (sizeof(T) * D > 256) ? 32 : 64;
  static constexpr int CH = TN * Tile<T, D>::CPR;          // chunks of a tile
  static constexpr int KB = TN / 32;
};

// Softmax state of a lane's row: the score, in base 2, that weights are relative to (-inf: nothing
// seen yet), and this lane's half of the sum of weights.
struct Row { float base = -INFINITY, l = 0.f; };

// One tile's softmax: s becomes the weights 2^{scale log2(e) s - base}.  The base follows the
// maximum when that has grown by over 8: weights stay below 2^8, and most tiles neither exchange
// maxima between the row's two lanes nor rescale.
template <int KB, int CB>
__device__ __forceinline__ void weigh(f16v (&s)[KB], float sc, Row &r, f16v (&acc)[CB]) {
  float top = s[0][0];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
  if (__any(fmaf(top, sc, -r.base) > 8.f)) {
    const float now = fmaxf(max_xor32(top) * sc, r.base);
    const float f = now == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(r.base - now);
    r.l *= f;
#pragma unroll
    for (int b = 0; b < CB; ++b) acc[b] *= f;
    r.base = now;
  }
  const float base = r.base == -INFINITY ? 0.f : r.base;
  float sum = 0.f;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[kb][i] = __builtin_amdgcn_exp2f(fmaf(s[kb][i], sc, -base));
      sum += s[kb][i];
    }
  r.l += sum;
}

// acc += V^T P^T for one tile of KB * 32 keys.
template <typename T, int D, int KB>
__device__ __forceinline__ void add_values(f16v (&acc)[D / 32], const f16v (&s)[KB], const uint4 *sv, int lane) {
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int b16 = 0; b16 < 2; ++b16) {
      const Frag<T> pf = result_frag<T>(s[kb], b16);
#pragma unroll
      for (int b = 0; b < D / 32; ++b) mma(acc[b], Tile<T, D>::cols(sv, kb * 32 + b16 * 16, b * 32, lane), pf);
    }
}

// Infinite and NaN values behind the mask.  A weight of 0 times one of them is not 0, so in a
// tile with keys that some rows do not see, or that ends behind the sequence's last key (which
// then stands there again, with weights of 0), they are set to 0 in LDS, and added afterwards, as
// they are, to the results of the rows that do see them: by the lane that wrote them (which
// reads its own writes; the sums are no longer in registers, so that this path costs the loop
// none), keys j0 .. j1 - 1.
template <typename T> __device__ __forceinline__ bool clean16(uint4 *p) {
  uint4v u = *reinterpret_cast<const uint4v *>(p);
  if (!nonfinite(u, T())) return false;
  *reinterpret_cast<uint4v *>(p) = only_finite(u, T());
  return true;
}
template <typename T, typename O, int D>
__device__ __forceinline__ void add_nonfinite(O *out, const T *v, int64_t ld, int j0, int j1, int h) {
#pragma unroll 1
  for (int j = j0; j < j1; ++j)
#pragma unroll 1
    for (int e = 4 * h; e < D; e += 8) {
      const f4 x = to_f4(ld4(v + j * ld + e));
      f4 o = to_f4(ld4(out + e));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(fabsf(x[i]) < INFINITY)) o[i] += x[i];
      store4(out + e, o[0], o[1], o[2], o[3]);
    }
}

// A lane's row: the result and lse, or, of one of several splits, the unnormalised sum [split]
// [row of the packed axis and head][d], then (reference in base 2, sum of weights).
template <typename T, int D>
__device__ __forceinline__ void finish(const AttnArgs &a, size_t at, int split, int h, float base, float l,
                                       const f16v (&acc)[D / 32]) {
  if (a.splits > 1) {
    const size_t nrow = (size_t)query_tokens(a) * a.hq, ps = split * nrow + at;
    float *p = a.part + ps * D;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        store4(p + b * 32 + 2 * i + 4 * h, acc[b][i], acc[b][i + 1], acc[b][i + 2], acc[b][i + 3]);
    if (h == 0) {
      float *ml = a.part + a.splits * nrow * D + ps * 2;
      ml[0] = base;
      ml[1] = l;
    }
    return;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
  T *out = static_cast<T *>(a.out) + at * D;
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      store4(out + b * 32 + 2 * i + 4 * h, acc[b][i] * inv, acc[b][i + 1] * inv, acc[b][i + 2] * inv,
             acc[b][i + 3] * inv);
  if (h == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (base + __builtin_amdgcn_logf(l));
}

template <typename T, int D>
__device__ __forceinline__ void restore(const AttnArgs &a, size_t at, int split, const T *v, int j0, int j1, int h) {
  if (a.splits > 1)
    add_nonfinite<T, float, D>(a.part + (split * (size_t)query_tokens(a) * a.hq + at) * D, v, a.ldv, j0, j1, h);
  else
    add_nonfinite<T, T, D>(static_cast<T *>(a.out) + at * D, v, a.ldv, j0, j1, h);
}

template <typename T, int D>
__global__ __launch_bounds__(THR, sizeof(T) * D > 256 ? 1 : sizeof(T) * D > 128 ? 2 : 4) void attn_fwd(AttnArgs a) {
  typedef Fwd<T, D> F;
  typedef Tile<T, D> Ti;
  constexpr int TN = F::TN, DB = D / 16, CB = D / 32;
  __shared__ uint4 sk[2][F::CH], sv[2][F::CH];
  __shared__ int sbad;                          // a value was cleaned
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, c = lane & 31, h = lane >> 5;

  // key head fastest (a head stays on one die where 8 and hk divide one another), then the
  // split of the keys, then the tiles
  unsigned id = blockIdx.x;
  const int head = id % (unsigned)a.hk;
  id /= (unsigned)a.hk;
  const int split = id % (unsigned)a.splits;
  id /= (unsigned)a.splits;
  int n, tile;
  if (a.cuq) {
    const Slot s = find_slot(a.cuq, a.n, id, a.group, TM);
    n = s.n;
    tile = s.tile;
  } else {
    n = id % (unsigned)a.n;
    tile = id / (unsigned)a.n;
  }
  const Seq q = seq_of(a, n);
  const int rows = q.Lq * a.group, tiles = (rows + TM - 1) / TM;
  if ((unsigned)tile >= (unsigned)tiles) return;
  tile = tiles - 1 - tile;                      // the tiles with the most keys start first

  const int off = q.Lk - q.Lq, r0 = tile * TM + wave * 32;
  const int r = min(r0 + c, rows - 1);
  const bool on = r0 + c < rows;
  const int tok = r / (unsigned)a.group, hq = head * a.group + (r - tok * a.group);
  const int lim = tok + off;                    // the last key this row sees
  const int first_lim = (int)((unsigned)min(r0, rows - 1) / (unsigned)a.group) + off;
  const int tile_lim = (int)((unsigned)(tile * TM) / (unsigned)a.group) + off;
  const int wave_lim = (int)((unsigned)min(r0 + 31, rows - 1) / (unsigned)a.group) + off;
  const int last_lim = (int)((unsigned)min(tile * TM + TM - 1, rows - 1) / (unsigned)a.group) + off;
  const int keys = max(min(q.Lk, last_lim + 1), 0), ktiles = (keys + TN - 1) / TN;
  const int kt0 = (int)((int64_t)ktiles * split / a.splits), kt1 = (int)((int64_t)ktiles * (split + 1) / a.splits);

  const T *qrow = static_cast<const T *>(a.q) + (int64_t)(q.q0 + tok) * a.ldq + hq * D;
  Frag<T> qf[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) qf[b] = global_frag(qrow, b, h);

  // Copying tiles.  Rows past the sequence's keys repeat its last one: no row of another
  // sequence is read, and their weights are 0.
  typedef Copy<T, D, TN> Cp;
  if (tid == 0) sbad = 0;
  __syncthreads();                              // before any wave sets it
  const T *kg = static_cast<const T *>(a.k) + (int64_t)q.k0 * a.ldk + head * D;
  const T *vg = static_cast<const T *>(a.v) + (int64_t)q.k0 * a.ldv + head * D;
  const unsigned kstep = (unsigned)a.ldk * sizeof(T), vstep = (unsigned)a.ldv * sizeof(T);
  unsigned ko[Cp::PER], vo[Cp::PER];
#pragma unroll
  for (int i = 0; i < Cp::PER; ++i) {
    ko[i] = Cp::row(i, tid) * kstep + Cp::byte(i, tid);
    vo[i] = Cp::row(i, tid) * vstep + Cp::byte(i, tid);
  }
  auto copy = [&](int kt, int buf) {
    const T *kp = kg + (int64_t)kt * TN * a.ldk, *vp = vg + (int64_t)kt * TN * a.ldv;
    const int last = q.Lk - 1 - kt * TN;
#pragma unroll
    for (int i = 0; i < Cp::PER; ++i) {
      if (!Cp::has(i, wave)) continue;
      unsigned kb = ko[i], vb = vo[i];
      if (last < TN - 1) {                      // the sequence's last tile
        const int row = min(Cp::row(i, tid), last);
        kb = row * kstep + Cp::byte(i, tid);
        vb = row * vstep + Cp::byte(i, tid);
      }
      copy_to_lds(kp, kb, Cp::to(sk[buf], i, wave));
      copy_to_lds(vp, vb, Cp::to(sv[buf], i, wave));
    }
  };

  // From tile hidden0 on, tiles have keys that some row of this tile does not see, or that stand in
  // for keys past the sequence's last; every wave cleans the values that it copied, before the
  // barrier that hands the tile over.
  const int hidden0 = max(tile_lim + 1, 0) / TN;
  auto clean = [&](int kt, int buf) {
    if (kt < hidden0) return;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < Cp::PER; ++i)
      if (Cp::has(i, wave)) bad |= clean16<T>(&sv[buf][256 * i + tid]);
    if (__any(bad) && lane == 0) sbad = 1;
  };

  const float sc = a.scale * kLog2e;
  f16v acc[CB];
  Row row;
#pragma unroll
  for (int b = 0; b < CB; ++b) acc[b] = zero16();
  if (kt0 < kt1) copy(kt0, 0);
  copies_done();
#pragma unroll
  for (int b = 0; b < DB; ++b) arrived(qf[b]);
  if (kt0 < kt1) clean(kt0, 0);
  __syncthreads();
  for (int kt = kt0; kt < kt1; ++kt) {
    const int buf = (kt - kt0) & 1;
    if (kt + 1 < kt1) copy(kt + 1, buf ^ 1);    // its last readers are behind the barrier
    if (kt * TN <= wave_lim) {                  // else no row of this wave sees a key of the tile
      f16v s[F::KB];
#pragma unroll
      for (int kb = 0; kb < F::KB; ++kb) {
        s[kb] = zero16();
#pragma unroll
        for (int b = 0; b < DB; ++b) mma(s[kb], Ti::rows(sk[buf], kb * 32, b, lane), qf[b]);
      }
      if (kt * TN + TN - 1 > first_lim) {       // the same for the whole wave
        const int left = lim - kt * TN - 4 * h; // key 8 (i / 4) + 4 h + i % 4 of the tile is seen up to here
#pragma unroll
        for (int kb = 0; kb < F::KB; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (kb * 32 + 8 * (i / 4) + (i & 3) > left) s[kb][i] = -INFINITY;
      }
      weigh<F::KB, CB>(s, sc, row, acc);
      add_values<T, D, F::KB>(acc, s, sv[buf], lane);
    }
    copies_done();
    if (kt + 1 < kt1) clean(kt + 1, buf ^ 1);
    __syncthreads();
  }
  const float l = add_xor32(row.l);
  if (!on) return;
  const size_t at = (size_t)(q.q0 + tok) * a.hq + hq;
  finish<T, D>(a, at, split, h, row.base, l, acc);
  if (sbad) restore<T, D>(a, at, split, vg, max(kt0, hidden0) * TN, min(lim + 1, kt1 * TN), h);
}

// ---- Few rows ------------------------------------------------------------------
// Single tokens and the like: at most 32 rows (of the average sequence and key head) meet long
// keys, and the time is that of reading K and V once.  A workgroup is one wave with its own 32
// rows, one split of the keys, tiles of 32 keys and its own part of LDS, so nothing waits at a
// barrier: tile t + 1 is on its way while tile t is used.
// 16 sequences of up to 16384 keys, 16 / 4 heads of 128, single tokens: 67 us for 329 MB (4.9 TB/s), and
// 5 us for the join.
constexpr int FEW = 32;

template <typename T, int D> __global__ __launch_bounds__(64, sizeof(T) * D > 256 ? 1 : 2) void attn_few(AttnArgs a) {
  typedef Tile<T, D> Ti;
  constexpr int TN = 32, CH = TN * Ti::CPR, PER = CH / 64, DB = D / 16, CB = D / 32;
  __shared__ uint4 sk[2][CH], sv[2][CH];
  const int lane = threadIdx.x, c = lane & 31, h = lane >> 5;
  unsigned id = blockIdx.x;
  const int head = id % (unsigned)a.hk;
  id /= (unsigned)a.hk;
  const int split = id % (unsigned)a.splits;
  id /= (unsigned)a.splits;
  int n, tile;
  if (a.cuq) {
    const Slot s = find_slot(a.cuq, a.n, id, a.group, FEW);
    n = s.n;
    tile = s.tile;
  } else {
    n = id % (unsigned)a.n;
    tile = id / (unsigned)a.n;
  }
  const Seq q = seq_of(a, n);
  const int rows = q.Lq * a.group;
  if ((unsigned)tile >= (unsigned)((rows + FEW - 1) / FEW)) return;
  const int off = q.Lk - q.Lq, r0 = tile * FEW, r = min(r0 + c, rows - 1);
  const int tok = r / (unsigned)a.group, hq = head * a.group + (r - tok * a.group);
  const int lim = tok + off;
  const int first_lim = (int)((unsigned)r0 / (unsigned)a.group) + off;
  const int last_lim = (int)((unsigned)min(r0 + FEW - 1, rows - 1) / (unsigned)a.group) + off;
  const int keys = max(min(q.Lk, last_lim + 1), 0), ktiles = (keys + TN - 1) / TN;
  const int kt0 = __builtin_amdgcn_readfirstlane((int)((int64_t)ktiles * split / a.splits));
  const int kt1 = __builtin_amdgcn_readfirstlane((int)((int64_t)ktiles * (split + 1) / a.splits));

  const T *qrow = static_cast<const T *>(a.q) + (int64_t)(q.q0 + tok) * a.ldq + hq * D;
  Frag<T> qf[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) qf[b] = global_frag(qrow, b, h);
  const T *kg = static_cast<const T *>(a.k) + (int64_t)q.k0 * a.ldk + head * D;
  const T *vg = static_cast<const T *>(a.v) + (int64_t)q.k0 * a.ldv + head * D;
  const unsigned kstep = (unsigned)a.ldk * sizeof(T), vstep = (unsigned)a.ldv * sizeof(T);
  auto copy = [&](int kt, int buf) {            // rows past the sequence's keys repeat its last one
    const T *kp = kg + (int64_t)kt * TN * a.ldk, *vp = vg + (int64_t)kt * TN * a.ldv;
    const int last = q.Lk - 1 - kt * TN;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 64 + lane, row = e / Ti::CPR;
      const unsigned in = ((e % Ti::CPR) ^ Ti::swizzle(row)) * 16;
      copy_to_lds(kp, min(row, last) * kstep + in, lds_address(sk[buf] + i * 64));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 64 + lane, row = e / Ti::CPR;
      const unsigned in = ((e % Ti::CPR) ^ Ti::swizzle(row)) * 16;
      copy_to_lds(vp, min(row, last) * vstep + in, lds_address(sv[buf] + i * 64));
    }
  };
  const float sc = a.scale * kLog2e;
  f16v acc[CB];
  Row row;
  bool bad = false;                                        // a value was cleaned
  const int hidden0 = max(first_lim + 1, 0) / TN;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");         // from here on only copies are counted
#pragma unroll
  for (int b = 0; b < DB; ++b) arrived(qf[b]);
#pragma unroll
  for (int b = 0; b < CB; ++b) acc[b] = zero16();
  if (kt0 < kt1) copy(kt0, 0);
  for (int kt = kt0; kt < kt1; ++kt) {
    const int buf = (kt - kt0) & 1;
    if (kt + 1 < kt1) {
      copy(kt + 1, buf ^ 1);
      copies_done_but<2 * PER>();                          // this tile's are there
    } else {
      copies_done();
    }
    if (kt >= hidden0) {                                   // keys that some row does not see, or past the last
#pragma unroll
      for (int i = 0; i < PER; ++i) bad |= clean16<T>(&sv[buf][64 * i + lane]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    f16v s[1] = {zero16()};
#pragma unroll
    for (int b = 0; b < DB; ++b) mma(s[0], Ti::rows(sk[buf], 0, b, lane), qf[b]);
    if (kt * TN + TN - 1 > first_lim) {
      const int left = lim - kt * TN - 4 * h;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * (i / 4) + (i & 3) > left) s[0][i] = -INFINITY;
    }
    weigh<1, CB>(s, sc, row, acc);
    add_values<T, D, 1>(acc, s, sv[buf], lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // the buffer is read; the next copy may fill it
  }
  const float l = add_xor32(row.l);
  const bool cleaned = __any(bad);
  if (r0 + c >= rows) return;
  const size_t at = (size_t)(q.q0 + tok) * a.hq + hq;
  finish<T, D>(a, at, split, h, row.base, l, acc);
  if (cleaned) restore<T, D>(a, at, split, vg, max(kt0, hidden0) * TN, min(lim + 1, kt1 * TN), h);
}

// Joins the splits of a row, one workgroup a row: a thread forms the factor of one split (of at most
// THR; one thread after the other over 64 splits took 20 us), then
// D / 4 threads side by side add every GR-th split's sums, and the groups are added in order.
template <typename T, int D> __global__ __launch_bounds__(THR) void attn_join(AttnArgs a, size_t nrow) {
  constexpr int L = D / 4, GR = THR / L, WAVES = THR / 64;
  __shared__ float sm[WAVES], sl[WAVES], sf[THR];
  __shared__ f4 so[GR][L];
  const size_t row = blockIdx.x;
  if (a.cuq && row >= (size_t)max(a.cuq[a.n], 0) * a.hq) return;    // behind the last sequence
  const int t = threadIdx.x, wave = t >> 6, g = t / L, e = t % L;
  const float *ml = a.part + a.splits * nrow * D;
  float ms = -INFINITY, l = 0.f;
  if (t < a.splits) {
    ms = ml[(t * nrow + row) * 2];
    l = ml[(t * nrow + row) * 2 + 1];
  }
  float m = ms;
#pragma unroll
  for (int i = 32; i > 0; i /= 2) m = fmaxf(m, __shfl_xor(m, i));
  if ((t & 63) == 0) sm[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) m = fmaxf(m, sm[w]);
  const float f = ms == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms - m);   // nothing seen in this split
  sf[t] = f;
  l *= f;
#pragma unroll
  for (int i = 32; i > 0; i /= 2) l += __shfl_xor(l, i);
  if ((t & 63) == 0) sl[wave] = l;
  __syncthreads();
  f4 o = zero4();
#pragma unroll 8
  for (int s = g; s < a.splits; s += GR)
    o += sf[s] * *reinterpret_cast<const f4 *>(a.part + (s * nrow + row) * D + e * 4);
  so[g][e] = o;
  __syncthreads();
  if (g) return;
  for (int i = 1; i < GR; ++i) o += so[i][e];
  l = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) l += sl[w];
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  store4(static_cast<T *>(a.out) + row * D + e * 4, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  if (e == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(l));
}

// The same where a row has few splits: D / 4 threads a row add them one after the other (3 splits
// of 64 x 32 x 16 rows: 46 us for the call, 60 with a workgroup a row).
constexpr int FEW_SPLITS = 8;
template <typename T, int D> __global__ __launch_bounds__(THR) void attn_join_few(AttnArgs a, size_t nrow) {
  constexpr int L = D / 4, GR = THR / L;
  const size_t row = (size_t)blockIdx.x * GR + threadIdx.x / L;
  const int e = threadIdx.x % L;
  if (row >= nrow || (a.cuq && row >= (size_t)max(a.cuq[a.n], 0) * a.hq)) return;
  const float *ml = a.part + a.splits * nrow * D;
  float m = -INFINITY, l = 0.f;
  float ms[FEW_SPLITS], ls[FEW_SPLITS];
  f4 p[FEW_SPLITS], o = zero4();
#pragma unroll
  for (int s = 0; s < FEW_SPLITS; ++s) {
    const bool on = s < a.splits;
    const size_t at = (on ? s : 0) * nrow + row;
    ms[s] = on ? ml[at * 2] : -INFINITY;
    ls[s] = on ? ml[at * 2 + 1] : 0.f;
    p[s] = on ? *reinterpret_cast<const f4 *>(a.part + at * D + e * 4) : zero4();
  }
#pragma unroll
  for (int s = 0; s < FEW_SPLITS; ++s) m = fmaxf(m, ms[s]);
#pragma unroll
  for (int s = 0; s < FEW_SPLITS; ++s) {
    const float f = ms[s] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms[s] - m);
    l = fmaf(f, ls[s], l);
    o += f * p[s];
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  store4(static_cast<T *>(a.out) + row * D + e * 4, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  if (e == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(l));
}

// Whether a sequence's rows (the average's) fit a single wave.  16 sequences of up to 16384 keys, 4
// rows: 67 us this way, 75 by attn_fwd; 8 x 2048 keys, 12 heads of 64, 1 and 32 rows: 13.8 and 16.7
// against 17.3 and 18.4.  64 rows, two waves that read the keys each: 119 us against 62 (16 x 8192).
bool few_rows(const AttnArgs &a) { return query_tokens(a) * a.group <= (int64_t)FEW * a.n; }

// Tiles of the packed row axis, at most; exact without cu.
int64_t slots_of(const AttnArgs &a) {
  const int tm = few_rows(a) ? FEW : TM;
  if (a.cuq) return (int64_t)a.Tq * a.group / tm + a.n;
  return ((int64_t)a.Tq * a.group + tm - 1) / tm * a.n;
}

// Splits of the keys: only where the tiles leave compute units idle, and at least so many keys (of
// the average sequence) a split that joining stays cheap beside them.
// Few rows: one wave a workgroup, so 2560 of them (5 stand on a compute unit, dealt twice over:
// 16 sequences of up to 16384 keys, 4 key heads of 128, took 98 us at 640 workgroups, 80 us at
// 1280 and 2560), or, where the rows' partial sums would be over a sixteenth of the keys and values,
// as many splits as that allows, down to 512 workgroups (32 rows on 16 x 8192 keys: 32 splits 77 us,
// 8 splits 58 us; 8 rows on 8 x 2048 keys of 12 heads: 8 splits 16 us, 2 splits 29 us).  At most
// 128: a single sequence of 65536 keys, 4 heads, took 35 us with 64 splits, 28 with 128 or 256.
// Other rows, bf16: a workgroup a compute unit and 512 keys (64 tokens on 4 x 8192 keys, 16 / 4 heads
// of 128: 35 us, at two workgroups a unit 41, unsplit 149; 4 x 512, 12 / 12 of 64, where 256
// keys a split would be two: 13 us unsplit, 20 split).  fp32, whose products take 8 times as long
// beside the same partial sums: two a unit and 256 keys (1 x 2048, 16 / 4 of 128: 187 us, at one
// a unit 311; 1 x 1024, 12 / 12 of 64: 40 us, with 512 keys 48, with 1024 80).
constexpr int MOST_SPLITS = 128;
int splits_of(bool bf16, const AttnArgs &a) {
  const bool few = few_rows(a);
  const int64_t blocks = (few ? a.n : slots_of(a)) * a.hk, keys = a.cuq ? a.Tk / a.n : a.Tk;
  int64_t s = few ? 2560 / blocks : bf16 ? (256 + blocks - 1) / blocks : 512 / blocks;
  if (few) {
    const int64_t rows = query_tokens(a) * a.group / a.n, least = 512 / blocks;
    const int64_t small = keys / (32 * (rows < 1 ? 1 : rows));
    if (s > small) s = small > least ? small : least;
  }
  const int64_t most = keys / (few || !bf16 ? 256 : 512);
  if (s > most) s = most;
  if (s > MOST_SPLITS) s = MOST_SPLITS;
  return s < 1 ? 1 : (int)s;
}

template <typename T, int D> hipError_t run(AttnArgs &a, hipStream_t s) {
  const int64_t blocks = slots_of(a) * a.hk * a.splits;
  const size_t nrow = (size_t)query_tokens(a) * a.hq;
  if (few_rows(a)) hipLaunchKernelGGL((attn_few<T, D>), dim3((unsigned)blocks), dim3(64), 0, s, a);
  else hipLaunchKernelGGL((attn_fwd<T, D>), dim3((unsigned)blocks), dim3(THR), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  constexpr int GR = THR / (D / 4);
  if (a.splits <= FEW_SPLITS)
    hipLaunchKernelGGL((attn_join_few<T, D>), dim3((unsigned)((nrow + GR - 1) / GR)), dim3(THR), 0, s, a, nrow);
  else
    hipLaunchKernelGGL((attn_join<T, D>), dim3((unsigned)nrow), dim3(THR), 0, s, a, nrow);
  return hipGetLastError();
}

}  // namespace

bool attn_fwd_fits(bool bf16, const AttnArgs &a) {   // the join too: splits only come with few rows
  return grid_fits(slots_of(a) * a.hk * splits_of(bf16, a), few_rows(a) ? 64 : THR);
}

size_t attn_fwd_workspace(bool bf16, int d, const AttnArgs &a) {
  const int s = splits_of(bf16, a);
  return s == 1 ? 0 : (size_t)s * query_tokens(a) * a.hq * (d + 2) * sizeof(float);
}

hipError_t launch_attn_fwd(bool bf16, int d, AttnArgs a, void *ws, hipStream_t s) {
  a.splits = splits_of(bf16, a);
  a.part = static_cast<float *>(ws);
#define FALCON_ATTN(D_) \
  if (d == D_) return bf16 ? run<__bf16, D_>(a, s) : run<float, D_>(a, s)
  FALCON_ATTN(32);
  FALCON_ATTN(64);
  FALCON_ATTN(128);
#undef FALCON_ATTN
  return hipErrorInvalidValue;
}

}  // namespace falcon
