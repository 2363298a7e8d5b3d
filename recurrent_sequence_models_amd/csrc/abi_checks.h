// Checks of arguments that the C ABI's sources share.  Host side only.
#pragma once
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "falcon.h"
#include "layer_kernels.h"

namespace falcon {
namespace abi {

inline bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool float_dtype(int d) { return d == FALCON_F32 || d == FALCON_BF16; }
inline int esize(int dtype) { return dtype == FALCON_F32 ? 4 : dtype == FALCON_BF16 ? 2 : 1; }

// A required (or, if null, optional) pointer with its alignment.
inline int need(const void *p, unsigned align) { return p && aligned(p, align) ? FALCON_OK : FALCON_ERR_INVALID_ARG; }
inline int maybe(const void *p, unsigned align) { return aligned(p, align) ? FALCON_OK : FALCON_ERR_INVALID_ARG; }

inline int status_of(hipError_t e) { return e == hipSuccess ? FALCON_OK : FALCON_ERR_HIP; }

inline int check_workspace(const void *ws, size_t have, size_t want) {
  if (want == 0) return FALCON_OK;
  if (!ws || have < want) return FALCON_ERR_WORKSPACE;
  return maybe(ws, 16);
}

// An output that is one of the inputs where others read those late.  (Partial overlaps are the caller's to avoid.)
inline int distinct(const void *out, const void *in) { return out && out == in ? FALCON_ERR_INVALID_ARG : FALCON_OK; }

inline int apart(const void *out, std::initializer_list<const void *> ins) {
  for (const void *in : ins)
    if (distinct(out, in) != FALCON_OK) return FALCON_ERR_INVALID_ARG;
  return FALCON_OK;
}

// An output that is an input of another stride: its tokens lie where others' inputs are.  (Of the same, for what is read
// token by token: an entry is read by the wave that writes it.)
inline int same_rows(const void *out, int64_t out_stride, const void *in, int64_t stride, int64_t tokens) {
  return tokens > 1 && stride != out_stride ? distinct(out, in) : FALCON_OK;
}

// [tokens, width] of entries of `e` bytes at a pointer with a token stride.
inline int check_rows(const void *p, int64_t stride, int64_t tokens, int64_t width, int e) {
  if (need(p, 16) != FALCON_OK || stride < width || stride > INT64_MAX / 16 / tokens || (stride * e) % 16 != 0)
    return FALCON_ERR_INVALID_ARG;
  return FALCON_OK;
}

}  // namespace abi
}  // namespace falcon

#define FALCON_TRY(x)                        \
  do {                                       \
    const int st_ = (x);                     \
    if (st_ != FALCON_OK) return st_;        \
  } while (0)
