// Internal launch interface of the operators of a state-space block (norm of the residual stream,
// short causal convolution, selective state-space scan, projections): between the C ABI
// (falcon_block_abi.cpp) and their kernels.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "layer_kernels.h"
#include "seq_plan.h"

namespace falcon {

inline size_t align16(size_t n) { return (n + 15) / 16 * 16; }

// out[c] = sum over i < rows of part[i][c], c < cols, in a fixed order; columns from `split` on go to
// out2[c - split].  Either output may be null.
hipError_t launch_column_sum(const float *part, int rows, int64_t cols, float *out, int64_t split, float *out2,
                             hipStream_t s);

// Norm of the residual stream.  Dense rows of `width` entries.
struct NormArgs {
  const void *x, *residual;      // forward: input, what it is added to or null; backward: x is the stream
  const float *w;                // [width] or null (ones)
  void *s, *y;                   // forward: stream or null, result; backward: y is dx
  float *scale;                  // [tokens], 8-bit results
  const void *dy, *ds;           // backward: incoming gradients of the result and (or null) of the stream
  float *part;                   // backward workspace: per-workgroup weight-gradient sums [blocks, width]
  int tokens, width, norm;
  float eps, inv_width;
};
size_t norm_bwd_workspace(bool bf16, int tokens, int width);
hipError_t launch_norm_fwd(bool bf16, bool q8, NormArgs a, hipStream_t s);
hipError_t launch_norm_bwd(bool bf16, NormArgs a, float *dw, void *ws, hipStream_t s);

// Short causal convolution.  x may have a token stride; the rest is dense.
struct ConvArgs {
  const void *x, *dy;            // [tokens, D]
  void *y, *dx;
  const float *w, *bias;         // [D, taps]; [D] or null
  const void *init, *d_final;    // [n, taps - 1, D] or null (zeros)
  void *final_state, *d_init;    // [n, taps - 1, D] or null
  float *part;                   // backward workspace: sums for the weights [blocks, D taps + D]
  SeqMap seq;
  int64_t ldx, lddx;
  int D, silu, run;              // run: tokens of a thread
};
bool conv_fits(bool bf16, SeqMap seq, int D);
bool conv_step_fits(bool bf16, int n, int D);
size_t conv_bwd_workspace(bool bf16, int taps, SeqMap seq, int D);
hipError_t launch_conv_fwd(bool bf16, int taps, ConvArgs a, hipStream_t s);
hipError_t launch_conv_bwd(bool bf16, int taps, ConvArgs a, float *dw, float *db, void *ws, hipStream_t s);
hipError_t launch_conv_step(bool bf16, int taps, ConvArgs a, hipStream_t s);

// Selective state-space scan.  x, dt, z [tokens, D] and B, C [tokens, N] may have token strides.
struct SsmArgs {
  const void *x, *dt, *z, *B, *C;   // z may be null
  const float *A, *skip, *bias;     // [D, N]; [D] or null; [D] or null
  const float *init;                // [n, D, N] or null (zeros); single tokens: the state
  float *final_state;               // [n, D, N] or null; single tokens: the new state
  void *y;                          // [tokens, D]
  float *states;                    // [chunks, D, N]: the state before every chunk, or null
  float *seg_map, *seg_state, *seg_sum;   // workspace, by segment: end state from zero, first state, sum of delta
  SeqMap seq;
  int64_t ldx, lddt, ldz, ldB, ldC;
  int D, softplus, seg;             // seg: tokens of a segment
  // backward: states is read; gradients of x, dt, z [tokens, D] and B, C [tokens, N], with token strides
  const void *dy;                   // [tokens, D]
  const float *d_final;             // [n, D, N] or null (zeros)
  void *dx, *ddt, *dz, *dB, *dC;
  float *d_init;                    // [n, D, N] or null
  float *part_bc, *part_A, *part_D; // workspace: sums by group of channels, by segment, by segment
  int64_t lddx, ldddt, lddz, lddB, lddC;
};
struct SsmGrads { float *dA, *dD, *dbias; };   // [D, N]; [D] or null; [D] or null
bool ssm_fits(SeqMap seq, int D, int N);
bool ssm_step_fits(int n, int D, int N);
size_t ssm_fwd_workspace(SeqMap seq, int D, int N);
hipError_t launch_ssm_fwd(bool bf16, int N, SsmArgs a, void *ws, hipStream_t s);
size_t ssm_bwd_workspace(SeqMap seq, int D, int N);
hipError_t launch_ssm_bwd(bool bf16, int N, SsmArgs a, SsmGrads o, void *ws, hipStream_t s);
hipError_t launch_ssm_step(bool bf16, int N, SsmArgs a, hipStream_t s);

// Projections.  A product out[j][i] = sum_k left(i, k) right(j, k), i < I, j < J, k < K, with its epilogue; `ld`:
// entries between two rows of memory.
constexpr int FALCON_SILU = 1, FALCON_GELU = 2;   // FALCON_ACT_*
struct LinearArgs {
  const void *left, *right;
  int64_t ldl, ldr, ldo;
  int I, J, K, splits;
  void *out;
  float *pre;                       // [J, I] or null
  const float *scale_l, *scale_r;   // [I], [J], of 8-bit operands
  const float *bias;                // [I] or null
  const void *residual;             // [J, I] or null
  float *part;                      // workspace: sums of the splits [splits, J, I]
  int act;
};
struct LinearGrads {
  const void *x, *w, *dy;           // [tokens, in], [out, in], [tokens, out]
  const float *pre;                 // [tokens, out], with an activation
  void *dx, *dw;                    // or null
  float *dbias;                     // or null
  int64_t ldx, lddy, lddx;
  int tokens, in, out, act;
};
bool linear_fits(int entry_bytes, int64_t tokens, int64_t in, int64_t out);
size_t linear_fwd_workspace(int entry_bytes, int64_t tokens, int64_t in, int64_t out);
size_t linear_bwd_workspace(int entry_bytes, bool act, int64_t tokens, int64_t in, int64_t out);
hipError_t launch_linear_fwd(int dtype, bool bf16_out, LinearArgs a, void *ws, hipStream_t s);
hipError_t launch_linear_bwd(bool bf16, const LinearGrads &g, void *ws, hipStream_t s);

}  // namespace falcon
