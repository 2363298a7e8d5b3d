// Tiles and fragments of the attention kernels for gfx950 (wave64).
//
// Every product is a 32x32 MFMA tile.  With lane l, c = l % 32, h = l / 32:
//   result (C-layout)   register i of 16 holds row 8 (i / 4) + 4 h + i % 4, column c
//   left operand        8 values a lane: row c of the left matrix, 16 summed indices
//   right operand       8 values a lane: column c of the right matrix, the same 16
// Which summed index stands in which of the 16 slots (h, j) is free as long as both
// operands agree, and two assignments are used:
//   along a row of memory      slot (h, j) = index 8 h + j: 16 contiguous bytes (bf16)
//   along a result's rows      slot (h, j) = row 4 h + j (j < 4), 8 + 4 h + j - 4 (j >= 4):
//                              registers 8 b .. 8 b + 7 of a result are, rounded, the
//                              right operand of a product that sums over its rows.
// So a product of scores feeds the next product from registers, without LDS; the other
// operand of that product is read from LDS by columns (transposing reads for bf16).
#pragma once
#include <hip/hip_runtime.h>

#include "lane_ops.h"
#include "layer_kernels.h"
#include "mfma_frag.h"

namespace falcon {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef unsigned int uint4v __attribute__((ext_vector_type(4)));

template <typename T> struct Frag;
template <> struct Frag<__bf16> { bf8 v; };
template <> struct Frag<float> { f4 lo, hi; };

__device__ __forceinline__ void mma(f16v &d, const Frag<__bf16> &a, const Frag<__bf16> &b) {
  d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, d, 0, 0, 0);
}
__device__ __forceinline__ void mma(f16v &d, const Frag<float> &a, const Frag<float> &b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_32x32x2f32(a.lo[j], b.lo[j], d, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_32x32x2f32(a.hi[j], b.hi[j], d, 0, 0, 0);
}
__device__ __forceinline__ f16v zero16() {
  f16v z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Registers 8 b .. 8 b + 7 of a result as a right operand.  bf16: each value is rounded to
// nearest even here, as the matrix product takes 8-bit mantissas; sums stay in fp32.
template <typename T> __device__ __forceinline__ Frag<T> result_frag(const f16v &x, int b);
template <> __device__ __forceinline__ Frag<__bf16> result_frag<__bf16>(const f16v &x, int b) {
  Frag<__bf16> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = (__bf16)x[8 * b + j];
  return f;
}
template <> __device__ __forceinline__ Frag<float> result_frag<float>(const f16v &x, int b) {
  return Frag<float>{f4{x[8 * b], x[8 * b + 1], x[8 * b + 2], x[8 * b + 3]},
                     f4{x[8 * b + 4], x[8 * b + 5], x[8 * b + 6], x[8 * b + 7]}};
}

// 8 values along a row of global memory (this lane's row, 16-entry block b).
__device__ __forceinline__ Frag<__bf16> global_frag(const __bf16 *row, int b, int h) {
  return {*reinterpret_cast<const bf8 *>(row + 16 * b + 8 * h)};
}
__device__ __forceinline__ Frag<float> global_frag(const float *row, int b, int h) {
  return {*reinterpret_cast<const f4 *>(row + 16 * b + 8 * h), *reinterpret_cast<const f4 *>(row + 16 * b + 8 * h + 4)};
}

__device__ __forceinline__ float dot(const Frag<__bf16> &a, const Frag<__bf16> &b) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf((float)a.v[j], (float)b.v[j], s);
  return s;
}
__device__ __forceinline__ float dot(const Frag<float> &a, const Frag<float> &b) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fmaf(a.lo[j], b.lo[j], s);
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fmaf(a.hi[j], b.hi[j], s);
  return s;
}

// Makes a fragment's loads arrive here.  The compiler waits for them at their first use, and where
// that is in a loop it waits there every time, for the loop's copies (below) as well, which it
// does not know of: the next tile's copies would be awaited as soon as they are issued.
__device__ __forceinline__ void arrived(Frag<__bf16> &f) { asm volatile("" : "+v"(f.v)); }
__device__ __forceinline__ void arrived(Frag<float> &f) { asm volatile("" : "+v"(f.lo), "+v"(f.hi)); }

// A tile of ROWS rows of D entries in LDS, in 16-byte chunks.  Chunk c of a row stands at
// place c ^ swizzle(row): reads of one chunk of 16 neighbouring rows, and column reads of
// 4 rows x 4 chunks, then touch all banks evenly (unswizzled, rows of 256 bytes put a
// column of chunks into one bank group).
template <typename T, int D> struct Tile {
  static constexpr int E = 16 / (int)sizeof(T);   // entries per chunk
  static constexpr int CPR = D / E;               // chunks per row
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (CPR >= 16) return ((row & 3) << 2) | ((row >> 2) & 3);
    if constexpr (CPR == 8) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    return (row >> 2) & 3;
  }
  static __device__ __forceinline__ int place(int row, int chunk) { return row * CPR + (chunk ^ swizzle(row)); }

  // Left operand: rows row0 + c, entries of 16-entry block b.
  static __device__ __forceinline__ Frag<T> rows(const uint4 *t, int row0, int b, int lane) {
    const int row = row0 + (lane & 31), h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      return {__builtin_bit_cast(bf8, t[place(row, 2 * b + h)])};
    } else {
      return {__builtin_bit_cast(f4, t[place(row, 4 * b + 2 * h)]), __builtin_bit_cast(f4, t[place(row, 4 * b + 2 * h + 1)])};
    }
  }
  // Left operand, transposed: columns col0 + c, rows row0 .. row0 + 15 in the result-row slots.
  static __device__ __forceinline__ Frag<T> cols(const uint4 *t, int row0, int col0, int lane) {
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      // a transposing read: lane j of 16 names 4 entries of row j / 4, and gets column j of the 4 x 16 block
      const int j = lane & 15, col = col0 + (lane & 16) + 4 * (j & 3);
      Frag<__bf16> f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = row0 + 8 * k + 4 * h + (j >> 2);
        const __bf16 *p = reinterpret_cast<const __bf16 *>(t + place(row, col / 8)) + (col & 7);
        const bf4 v = ldtr(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.v[4 * k + i] = v[i];
      }
      return f;
    } else {
      const int col = col0 + (lane & 31);
      const float *p = reinterpret_cast<const float *>(t);
      Frag<float> f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f.lo[i] = p[4 * place(row0 + 4 * h + i, col / 4) + (col & 3)];
        f.hi[i] = p[4 * place(row0 + 8 + 4 * h + i, col / 4) + (col & 3)];
      }
      return f;
    }
  }
};

// Which sequence and tile a slot of a packed axis is.  Sequence n's tiles of `per` rows
// (`mul` rows a token) start at slot cu[n] * mul / per + n, which no two sequences share
// (floor(a) + ceil(b) <= floor(a + b) + 1) and which the device finds from cu alone.
struct Slot { int n, tile; };
__device__ __forceinline__ Slot find_slot(const int *cu, int N, int slot, int mul, int per) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int)((int64_t)cu[mid] * mul / per) + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return Slot{lo, slot - ((int)((int64_t)cu[lo] * mul / per) + lo)};
}

// 16 bytes a lane from global memory (a scalar base plus 32 bits a lane) straight into LDS, lane
// l's to lds + 16 l.  The compiler does not count these: copies_done() before the barrier that
// hands the tile over.
__device__ __forceinline__ const void *scalar(const void *base) {   // the same in every lane; the compiler may not know
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return reinterpret_cast<const void *>((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)p) |
                                        (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(p >> 32)) << 32);
}
__device__ __forceinline__ void copy_to_lds(const void *base, unsigned offset, unsigned lds) {
  base = scalar(base);
  lds = __builtin_amdgcn_readfirstlane((int)lds);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(offset), "s"(base), "s"(lds)
               : "memory", "m0");
}
// The same for 4 bytes a lane, lane l's to lds + 4 l.
__device__ __forceinline__ void copy4_to_lds(const void *base, unsigned offset, unsigned lds) {
  base = scalar(base);
  lds = __builtin_amdgcn_readfirstlane((int)lds);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(offset), "s"(base), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void copies_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// All but the last N of this wave's copies; N at most 63, and only copies outstanding.
template <int N> __device__ __forceinline__ void copies_done_but() {
  static_assert(N <= 63, "the counter's range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ unsigned lds_address(const void *p) {
  return (unsigned)(size_t)(__attribute__((address_space(3))) const void *)p;
}

// The share of one thread of 256 in copying tiles of ROWS rows of D entries: PER pieces of 16
// bytes, piece i of wave w being the tile's places 64 (4 i + w) .. + 63.
template <typename T, int D, int ROWS> struct Copy {
  typedef Tile<T, D> Ti;
  static constexpr int CH = ROWS * Ti::CPR, PER = (CH + 255) / 256;
  static constexpr bool ALL = CH % 256 == 0;     // else the last waves have nothing to copy
  static __device__ __forceinline__ bool has(int i, int wave) { return ALL || 64 * (4 * i + wave) < CH; }
  static __device__ __forceinline__ int row(int i, int tid) { return (256 * i + tid) / Ti::CPR; }
  // bytes of the piece within its row: the chunk whose place this is
  static __device__ __forceinline__ unsigned byte(int i, int tid) {
    return (((256 * i + tid) % Ti::CPR) ^ Ti::swizzle(row(i, tid))) * 16;
  }
  static __device__ __forceinline__ unsigned to(const uint4 *tile, int i, int wave) {
    return lds_address(tile + 64 * (4 * i + wave));
  }
};

// Tokens of the packed axes, or of all sequences.
__host__ __device__ __forceinline__ int64_t query_tokens(const AttnArgs &a) {
  return a.cuq ? (int64_t)a.Tq : (int64_t)a.n * a.Tq;
}
__host__ __device__ __forceinline__ int64_t key_tokens(const AttnArgs &a) {
  return a.cuk ? (int64_t)a.Tk : (int64_t)a.n * a.Tk;
}

// A sequence's token ranges, kept inside the arrays whatever the offsets hold.
struct Seq { int q0, Lq, k0, Lk; };
__device__ __forceinline__ void clamp_range(const int *cu, int n, int total, int &begin, int &length) {
  begin = min(max(cu[n], 0), total);
  length = max(min(cu[n + 1], total) - begin, 0);
}
__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int n) {
  if (!a.cuq) return Seq{n * a.Tq, a.Tq, n * a.Tk, a.Tk};
  Seq s;
  clamp_range(a.cuq, n, a.Tq, s.q0, s.Lq);
  clamp_range(a.cuk, n, a.Tk, s.k0, s.Lk);
  return s;
}

// max with the lane 32 away, by the lane swap of lane_ops.h.  Every lane of the wave calls it.
__device__ __forceinline__ float max_xor32(float x) {
  float a = x, b = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(a), "+v"(b));
  return fmaxf(a, b);
}

// Whether any of 16 bytes of entries is infinite or NaN (exponent all ones).
__device__ __forceinline__ bool nonfinite(const uint4v &u, __bf16) {
  unsigned r = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) r |= (u[j] & 0x7fff7fffu) + 0x00800080u;
  return (r & 0x80008000u) != 0;
}
__device__ __forceinline__ bool nonfinite(const uint4v &u, float) {
  unsigned r = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) r |= (u[j] & 0x7fffffffu) + 0x00800000u;
  return (r & 0x80000000u) != 0;
}

// The same 16 bytes with zeros in their place.
__device__ __forceinline__ uint4v only_finite(uint4v u, __bf16) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const unsigned top = ((u[j] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;   // the top bit of a half that goes
    u[j] &= ~((top >> 15) * 0xffffu);
  }
  return u;
}
__device__ __forceinline__ uint4v only_finite(uint4v u, float) {
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = (u[j] & 0x7fffffffu) + 0x00800000u >= 0x80000000u ? 0u : u[j];
  return u;
}

// 4 consecutive results; bf16: rounded to nearest even.
__device__ __forceinline__ void store4(__bf16 *p, float a, float b, float c, float d) {
  *reinterpret_cast<bf4 *>(p) = __builtin_convertvector(f4{a, b, c, d}, bf4);
}
__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
  *reinterpret_cast<f4 *>(p) = f4{a, b, c, d};
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

}  // namespace falcon
