// Internal launch interface of the layer operators (gated linear recurrence,
// query / key norm with rotary positions, causal attention): between the C ABI
// (falcon_layer_abi.cpp) and their kernels.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace falcon {

// A launch holds less than 2^32 threads.
inline bool grid_fits(int64_t blocks, int threads) { return blocks >= 0 && blocks <= UINT32_MAX / threads; }

// Gated linear recurrence.  Packed calls (cu != null) have rows = 1 and T = the
// packed length; nseq sequences.  Otherwise rows = nseq sequences of T steps.
struct ScanArgs {
  const void *x, *g;             // [rows, T, D] in the input dtype
  const int *cu;                 // [nseq + 1] token offsets, or null
  const float *init;             // [nseq, D] or null (zeros)
  float *final_state;            // [nseq, D] or null
  void *h;                       // [rows, T, D]
  float *states;                 // [rows, NC, D]: h at the end of every chunk (backward: read), or null
  const void *dh;                // backward: [rows, T, D]
  const float *d_final;          // backward: [nseq, D] or null (zeros)
  void *dx, *dg;                 // backward: [rows, T, D]
  float *d_init;                 // backward: [nseq, D] or null
  unsigned int *ticket;          // workspace (NC > 1): one counter per column,
  unsigned long long *agg;       // one chunk map per (column, chunk, channel),
  unsigned long long *pre;       // one carry per (column, group of chunks, channel)
  int rows, T, D, nseq, NC;
};
bool scan_fits(bool bf16, int rows, int T, int D);          // within a launch
size_t scan_workspace(bool bf16, int rows, int T, int D);
hipError_t launch_scan_fwd(bool bf16, bool mix, ScanArgs a, void *ws, hipStream_t s);
hipError_t launch_scan_bwd(bool bf16, bool mix, ScanArgs a, void *ws, hipStream_t s);
hipError_t launch_scan_step(bool bf16, bool mix, const void *x, const void *g, float *state, void *h, size_t n,
                            hipStream_t s);

// Query / key norm with rotary positions.  Rows of a token are its heads; `ld` is the
// distance between tokens in elements (heads of a token are dense).
struct QkTensor { const void *p; int64_t ld; };
struct QkArgs {
  QkTensor x[2], y[2];           // forward: inputs, outputs; backward: inputs, gradients of the inputs
  QkTensor dy[2];                // backward: incoming gradients
  const float *w[2];             // [d] or null (ones)
  float *dw[2];                  // backward: [d] or null
  const int *pos;                // [tokens]
  const double *freq;            // [rot / 2]: radians per position
  float *part;                   // workspace: per-workgroup weight-gradient sums [blocks, 2, d]
  int tokens, hq, hk, rot, tok;  // tok: tokens of a workgroup at a time
  int norm, interleaved;
  float eps, scale;              // scale: factor of the rotated part
};
size_t qk_bwd_workspace(int tokens, int d);
hipError_t launch_qk_fwd(bool bf16, int d, QkArgs a, hipStream_t s);
hipError_t launch_qk_bwd(bool bf16, bool dy_f32, int d, QkArgs a, void *ws, hipStream_t s);

// Causal attention with grouped heads.  Packed calls have cuq and cuk; otherwise the
// sequences are Tq and Tk tokens each.  `ld`: elements between tokens.
struct AttnArgs {
  const void *q, *k, *v;         // [tokens, heads, d]
  const void *o, *d_o;           // backward
  const float *lse_in;           // backward
  void *out, *dq, *dk, *dv;
  float *lse;                    // [query tokens, hq]
  const int *cuq, *cuk;          // [n + 1] or null
  float *part;                   // workspace: partial results of splits
  float *delta, *lse2;           // backward workspace: -do . o and lse in base 2 of every row
  int64_t ldq, ldk, ldv, lddo, lddq, lddk, lddv;
  int n, Tq, Tk;                 // packed: Tq, Tk are the totals
  int hq, hk, group;             // group = hq / hk
  int splits;                    // filled at launch
  float scale;
};
bool attn_fwd_fits(bool bf16, const AttnArgs &a);           // within a launch
bool attn_bwd_fits(int d, const AttnArgs &a);
size_t attn_fwd_workspace(bool bf16, int d, const AttnArgs &a);
hipError_t launch_attn_fwd(bool bf16, int d, AttnArgs a, void *ws, hipStream_t s);
size_t attn_bwd_workspace(int d, const AttnArgs &a);
hipError_t launch_attn_bwd(bool bf16, int d, AttnArgs a, void *ws, hipStream_t s);

}  // namespace falcon
