// Rows of bf16 or fp32 entries, 16 bytes a lane, as the block operators read and write them.
#pragma once
#include <hip/hip_runtime.h>

#include "lane_ops.h"
#include "mfma_frag.h"

namespace falcon {

typedef unsigned int u4 __attribute__((ext_vector_type(4)));   // 16 bytes of entries, in registers

template <typename T> constexpr int PER16 = 16 / (int)sizeof(T);   // entries in 16 bytes

__device__ __forceinline__ void widen(const u4 &u, float (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[2 * j] = __uint_as_float(u[j] << 16);
    o[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const u4 &u, float (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = __uint_as_float(u[j]);
}
// Rounded to nearest even: the one rounding of a result held in bf16.
__device__ __forceinline__ u4 narrow(const float (&v)[8]) {
  bf8 b;
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = (__bf16)v[j];
  return __builtin_bit_cast(u4, b);
}
__device__ __forceinline__ u4 narrow(const float (&v)[4]) {
  return u4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}
template <typename T> __device__ __forceinline__ u4 load16(const T *p) { return *reinterpret_cast<const u4 *>(p); }
template <typename T> __device__ __forceinline__ void store16(T *p, const u4 &v) { *reinterpret_cast<u4 *>(p) = v; }
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

// V consecutive entries as they are in memory (whole registers, or half of one), at an address that is a multiple of
// their size together; for what is loaded long before its use.
template <typename T, int V> struct Few {
  static constexpr int BYTES = V * (int)sizeof(T), WORDS = BYTES < 4 ? 1 : BYTES / 4;
  unsigned u[WORDS];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[j]);
    return __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
  }
};
template <typename T, int V> __device__ __forceinline__ void fetch(const T *p, Few<T, V> &o) {
  if constexpr (Few<T, V>::BYTES == 16) {
    const u4 t = *reinterpret_cast<const u4 *>(p);
    o.u[0] = t[0]; o.u[1] = t[1]; o.u[2] = t[2]; o.u[3] = t[3];
  } else if constexpr (Few<T, V>::BYTES == 8) {
    const uint2 t = *reinterpret_cast<const uint2 *>(p);
    o.u[0] = t.x; o.u[1] = t.y;
  } else if constexpr (Few<T, V>::BYTES == 4) {
    o.u[0] = *reinterpret_cast<const unsigned *>(p);
  } else {
    static_assert(Few<T, V>::BYTES == 2, "1 to 16 bytes");
    o.u[0] = *reinterpret_cast<const unsigned short *>(p);
  }
}
template <typename T, int V> __device__ __forceinline__ void put(T *p, const Few<T, V> &o) {
  if constexpr (Few<T, V>::BYTES == 16) *reinterpret_cast<u4 *>(p) = u4{o.u[0], o.u[1], o.u[2], o.u[3]};
  else if constexpr (Few<T, V>::BYTES == 8) *reinterpret_cast<uint2 *>(p) = uint2{o.u[0], o.u[1]};
  else if constexpr (Few<T, V>::BYTES == 4) *reinterpret_cast<unsigned *>(p) = o.u[0];
  else *reinterpret_cast<unsigned short *>(p) = (unsigned short)o.u[0];
}
// Rounded to nearest even: the one rounding of a result held in bf16.
__device__ __forceinline__ void put(__bf16 *p, const float (&v)[8]) { store16(p, narrow(v)); }
__device__ __forceinline__ void put(float *p, const float (&v)[4]) { store16(p, narrow(v)); }
__device__ __forceinline__ void put(__bf16 *p, const float (&v)[4]) {
  *reinterpret_cast<bf4 *>(p) = __builtin_convertvector(f4{v[0], v[1], v[2], v[3]}, bf4);
}
__device__ __forceinline__ void put(float *p, const float (&v)[2]) { *reinterpret_cast<float2 *>(p) = float2{v[0], v[1]}; }
__device__ __forceinline__ void put(__bf16 *p, const float (&v)[2]) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  *reinterpret_cast<bf2 *>(p) = bf2{(__bf16)v[0], (__bf16)v[1]};
}
template <typename T> __device__ __forceinline__ void put(T *p, const float (&v)[1]) { *p = (T)v[0]; }

// Sum over the 64 lanes of a wave, in each of them.
__device__ __forceinline__ float wave_sum(float x) { return add_xor32(add_xor16(lane_sum<16>(x))); }
// The largest of 64 lanes' unsigned values, in each of them.
__device__ __forceinline__ unsigned wave_max(unsigned x) {
#pragma unroll
  for (int k = 1; k < 64; k *= 2) x = max(x, (unsigned)__shfl_xor((int)x, k));
  return x;
}

// 1 / (1 + e^-v) by the hardware's exp2 and reciprocal (each within one step): exact 0 and 1 at the ends, as
// e^-v becomes infinite or 0 there.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.44269504088896f));
}

}  // namespace falcon
