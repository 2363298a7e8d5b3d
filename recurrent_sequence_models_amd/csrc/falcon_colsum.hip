// Sums of partial results over workgroups, in a fixed order: the last step of the gradients of
// parameters, out[c] = sum over i < rows of part[i][c].
//
// 16 columns and 64 slices of the rows a workgroup; each slice's sum is sequential, and so is the sum of
// the slices.
#include "block_kernels.h"

namespace falcon {
namespace {

constexpr int COLS = 16, SLICES = 1024 / COLS;

__global__ __launch_bounds__(1024) void column_sum(const float *part, int rows, int64_t cols, float *out, int64_t split,
                                                   float *out2) {
  __shared__ float sum[SLICES][COLS];
  const int e = threadIdx.x % COLS, sl = threadIdx.x / COLS;
  const int64_t c = (int64_t)blockIdx.x * COLS + e;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int i = sl; i < rows; i += SLICES) s += part[(size_t)i * cols + c];
  }
  sum[sl][e] = s;
  __syncthreads();
  if (threadIdx.x < COLS && c < cols) {
    s = 0.f;
#pragma unroll 8
    for (int i = 0; i < SLICES; ++i) s += sum[i][e];
    float *to = c < split ? out : out2;
    if (to) to[c < split ? c : c - split] = s;
  }
}

}  // namespace

hipError_t launch_column_sum(const float *part, int rows, int64_t cols, float *out, int64_t split, float *out2,
                             hipStream_t s) {
  hipLaunchKernelGGL(column_sum, dim3((unsigned)((cols + COLS - 1) / COLS)), dim3(1024), 0, s, part, rows, cols, out, split,
                     out2);
  return hipGetLastError();
}

}  // namespace falcon
