// C ABI of the layer operators (declared in include/falcon.h): the gated linear
// recurrence, the query / key norm with rotary positions, and causal attention.
//
// Host side only, as falcon_abi.cpp: every argument is validated before the first HIP
// call.  The kernels live in falcon_scan.hip, falcon_qk.hip, falcon_attn.hip and
// falcon_attn_bwd.hip.
#include "falcon.h"

#include <cmath>
#include <cstdint>

#include "layer_kernels.h"

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int d) { return d == FALCON_F32 || d == FALCON_BF16; }
int esize(int dtype) { return dtype == FALCON_BF16 ? 2 : 4; }

// A required (or, if null, optional) pointer with its alignment.
int need(const void *p, unsigned align) { return p && aligned(p, align) ? FALCON_OK : FALCON_ERR_INVALID_ARG; }
int maybe(const void *p, unsigned align) { return aligned(p, align) ? FALCON_OK : FALCON_ERR_INVALID_ARG; }

int status_of(hipError_t e) { return e == hipSuccess ? FALCON_OK : FALCON_ERR_HIP; }

int check_workspace(const void *ws, size_t have, size_t want) {
  if (want == 0) return FALCON_OK;
  if (!ws || have < want) return FALCON_ERR_WORKSPACE;
  return maybe(ws, 16);
}

}  // namespace

#define FALCON_TRY(x)                        \
  do {                                       \
    const int st_ = (x);                     \
    if (st_ != FALCON_OK) return st_;        \
  } while (0)

// ---- Gated linear recurrence ---------------------------------------------------
namespace {

int check_scan(const falcon_scan_shape_t *s, bool packed, bool step) {
  if (!s || !dtype_ok(s->dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->input != FALCON_SCAN_ADD && s->input != FALCON_SCAN_MIX) return FALCON_ERR_INVALID_ARG;
  if (s->batch < 1 || s->width < 1 || (!step && s->seqlen < 1)) return FALCON_ERR_INVALID_ARG;
  if (s->width % 8 != 0 || s->width > (1 << 20)) return FALCON_ERR_UNSUPPORTED;
  if (step) {
    const int64_t threads = (int64_t)s->batch * s->width * esize(s->dtype) / 16;
    return falcon::grid_fits((threads + 255) / 256, 256) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
  }
  // step and sequence numbers are ints, with a chunk or a stride over the sequences added
  if (s->seqlen > INT32_MAX - FALCON_SCAN_CHUNK || s->batch > (1 << 30)) return FALCON_ERR_UNSUPPORTED;
  return falcon::scan_fits(s->dtype == FALCON_BF16, packed ? 1 : s->batch, s->seqlen, s->width) ? FALCON_OK
                                                                                                : FALCON_ERR_UNSUPPORTED;
}

falcon::ScanArgs scan_args(const falcon_scan_shape_t *s, const int32_t *cu, const void *x, const void *g,
                           const float *init) {
  falcon::ScanArgs a{};
  a.x = x;
  a.g = g;
  a.cu = cu;
  a.init = init;
  a.rows = cu ? 1 : s->batch;
  a.T = s->seqlen;
  a.D = s->width;
  a.nseq = s->batch;
  return a;
}

}  // namespace

extern "C" {

size_t falcon_scan_workspace(const falcon_scan_shape_t *s, int packed) {
  if (check_scan(s, packed != 0, false) != FALCON_OK) return 0;
  return falcon::scan_workspace(s->dtype == FALCON_BF16, packed ? 1 : s->batch, s->seqlen, s->width);
}

int falcon_scan_fwd(const falcon_scan_shape_t *s, const int32_t *cu, const void *x, const void *g, const float *init,
                    float *final_state, void *h, float *chunk_states, void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_scan(s, cu != nullptr, false));
  FALCON_TRY(maybe(cu, 4));
  FALCON_TRY(need(x, 16));
  FALCON_TRY(need(g, 16));
  FALCON_TRY(need(h, 16));
  FALCON_TRY(maybe(init, 16));
  FALCON_TRY(maybe(final_state, 16));
  FALCON_TRY(maybe(chunk_states, 16));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_scan_workspace(s, cu != nullptr)));
  falcon::ScanArgs a = scan_args(s, cu, x, g, init);
  a.final_state = final_state;
  a.h = h;
  a.states = chunk_states;
  return status_of(falcon::launch_scan_fwd(s->dtype == FALCON_BF16, s->input == FALCON_SCAN_MIX, a, ws,
                                           static_cast<hipStream_t>(stream)));
}

int falcon_scan_bwd(const falcon_scan_shape_t *s, const int32_t *cu, const void *x, const void *g, const float *init,
                    const float *chunk_states, const void *d_h, const float *d_final, void *dx, void *dg, float *d_init,
                    void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_scan(s, cu != nullptr, false));
  FALCON_TRY(maybe(cu, 4));
  FALCON_TRY(need(x, 16));
  FALCON_TRY(need(g, 16));
  FALCON_TRY(need(d_h, 16));
  FALCON_TRY(need(dx, 16));
  FALCON_TRY(need(dg, 16));
  FALCON_TRY(need(chunk_states, 16));
  FALCON_TRY(maybe(init, 16));
  FALCON_TRY(maybe(d_final, 16));
  FALCON_TRY(maybe(d_init, 16));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_scan_workspace(s, cu != nullptr)));
  falcon::ScanArgs a = scan_args(s, cu, x, g, init);
  a.states = const_cast<float *>(chunk_states);
  a.dh = d_h;
  a.d_final = d_final;
  a.dx = dx;
  a.dg = dg;
  a.d_init = d_init;
  return status_of(falcon::launch_scan_bwd(s->dtype == FALCON_BF16, s->input == FALCON_SCAN_MIX, a, ws,
                                           static_cast<hipStream_t>(stream)));
}

int falcon_scan_step(const falcon_scan_shape_t *s, const void *x, const void *g, float *state, void *h, void *stream) {
  FALCON_TRY(check_scan(s, false, true));
  FALCON_TRY(need(x, 16));
  FALCON_TRY(need(g, 16));
  FALCON_TRY(need(state, 16));
  FALCON_TRY(need(h, 16));
  return status_of(falcon::launch_scan_step(s->dtype == FALCON_BF16, s->input == FALCON_SCAN_MIX, x, g, state, h,
                                            (size_t)s->batch * s->width, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- Heads ---------------------------------------------------------------------
namespace {

// [tokens, heads, d] of entries of `e` bytes at a pointer with a token stride.
int check_heads(const void *p, int64_t stride, int64_t tokens, int64_t heads, int d, int e) {
  FALCON_TRY(need(p, 16));
  if (stride < heads * d || (stride * e) % 16 != 0) return FALCON_ERR_INVALID_ARG;
  if (stride > INT64_MAX / 16 / tokens) return FALCON_ERR_INVALID_ARG;
  return FALCON_OK;
}
int check_d(int d) { return d == 32 || d == 64 || d == 128 ? FALCON_OK : FALCON_ERR_UNSUPPORTED; }

// ---- Query / key norm with rotary positions --------------------------------------
int check_qk(const falcon_qk_shape_t *s) {
  if (!s || !dtype_ok(s->dtype) || !dtype_ok(s->grad_dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->tokens < 1 || s->heads_q < 1 || s->heads_k < 1 || s->d < 1) return FALCON_ERR_INVALID_ARG;
  if (s->layout != FALCON_ROPE_HALF && s->layout != FALCON_ROPE_INTERLEAVED) return FALCON_ERR_INVALID_ARG;
  if (s->norm != 0 && s->norm != 1) return FALCON_ERR_INVALID_ARG;
  if (!std::isfinite(s->eps) || s->eps < 0.f || !std::isfinite(s->rot_scale)) return FALCON_ERR_INVALID_ARG;
  if (s->rot < 0 || s->rot > s->d) return FALCON_ERR_INVALID_ARG;
  FALCON_TRY(check_d(s->d));
  if (s->rot % 16 != 0) return FALCON_ERR_UNSUPPORTED;
  // the rows of a workgroup's tokens, and token numbers past the last, are ints
  if ((int64_t)s->heads_q + s->heads_k > (1 << 20) || s->tokens > INT32_MAX - (1 << 20)) return FALCON_ERR_UNSUPPORTED;
  return FALCON_OK;
}

int check_qk_common(const falcon_qk_shape_t *s, const float *wq, const float *wk, const int32_t *pos,
                    const double *freq) {
  FALCON_TRY(maybe(wq, 16));
  FALCON_TRY(maybe(wk, 16));
  FALCON_TRY(s->rot ? need(freq, 8) : maybe(freq, 8));
  return need(pos, 4);
}

falcon::QkArgs qk_args(const falcon_qk_shape_t *s, const float *wq, const float *wk, const int32_t *pos,
                       const double *freq) {
  falcon::QkArgs a{};
  a.w[0] = s->norm ? wq : nullptr;
  a.w[1] = s->norm ? wk : nullptr;
  a.pos = pos;
  a.freq = freq;
  a.tokens = s->tokens;
  a.hq = s->heads_q;
  a.hk = s->heads_k;
  a.rot = s->rot;
  a.norm = s->norm;
  a.interleaved = s->layout == FALCON_ROPE_INTERLEAVED;
  a.eps = s->eps;
  a.scale = s->rot_scale;
  return a;
}

}  // namespace

extern "C" {

int falcon_qk_norm_rope(const falcon_qk_shape_t *s, falcon_heads_t q, falcon_heads_t k, const float *wq, const float *wk,
                        const int32_t *pos, const double *freq, falcon_heads_out_t qo, falcon_heads_out_t ko,
                        void *stream) {
  FALCON_TRY(check_qk(s));
  FALCON_TRY(check_qk_common(s, wq, wk, pos, freq));
  const int e = esize(s->dtype);
  FALCON_TRY(check_heads(q.data, q.token_stride, s->tokens, s->heads_q, s->d, e));
  FALCON_TRY(check_heads(k.data, k.token_stride, s->tokens, s->heads_k, s->d, e));
  FALCON_TRY(check_heads(qo.data, qo.token_stride, s->tokens, s->heads_q, s->d, e));
  FALCON_TRY(check_heads(ko.data, ko.token_stride, s->tokens, s->heads_k, s->d, e));
  falcon::QkArgs a = qk_args(s, wq, wk, pos, freq);
  a.x[0] = {q.data, q.token_stride};
  a.x[1] = {k.data, k.token_stride};
  a.y[0] = {qo.data, qo.token_stride};
  a.y[1] = {ko.data, ko.token_stride};
  return status_of(falcon::launch_qk_fwd(s->dtype == FALCON_BF16, s->d, a, static_cast<hipStream_t>(stream)));
}

size_t falcon_qk_norm_rope_bwd_workspace(const falcon_qk_shape_t *s) {
  if (check_qk(s) != FALCON_OK || !s->norm) return 0;
  return falcon::qk_bwd_workspace(s->tokens, s->d);
}

int falcon_qk_norm_rope_bwd(const falcon_qk_shape_t *s, falcon_heads_t q, falcon_heads_t k, const float *wq,
                            const float *wk, const int32_t *pos, const double *freq, falcon_heads_t dqo,
                            falcon_heads_t dko, falcon_heads_out_t dq, falcon_heads_out_t dk, float *dwq, float *dwk,
                            void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_qk(s));
  if (s->grad_dtype != s->dtype && s->grad_dtype != FALCON_F32) return FALCON_ERR_UNSUPPORTED;
  FALCON_TRY(check_qk_common(s, wq, wk, pos, freq));
  const int e = esize(s->dtype), eg = esize(s->grad_dtype);
  if (s->norm) {
    FALCON_TRY(check_heads(q.data, q.token_stride, s->tokens, s->heads_q, s->d, e));
    FALCON_TRY(check_heads(k.data, k.token_stride, s->tokens, s->heads_k, s->d, e));
  }
  FALCON_TRY(check_heads(dqo.data, dqo.token_stride, s->tokens, s->heads_q, s->d, eg));
  FALCON_TRY(check_heads(dko.data, dko.token_stride, s->tokens, s->heads_k, s->d, eg));
  FALCON_TRY(check_heads(dq.data, dq.token_stride, s->tokens, s->heads_q, s->d, e));
  FALCON_TRY(check_heads(dk.data, dk.token_stride, s->tokens, s->heads_k, s->d, e));
  FALCON_TRY(maybe(dwq, 4));
  FALCON_TRY(maybe(dwk, 4));
  if (!s->norm && (dwq || dwk)) return FALCON_ERR_INVALID_ARG;   // no weights, no gradients of them
  if (dwq || dwk) FALCON_TRY(check_workspace(ws, ws_bytes, falcon_qk_norm_rope_bwd_workspace(s)));
  falcon::QkArgs a = qk_args(s, wq, wk, pos, freq);
  a.x[0] = {q.data, q.token_stride};
  a.x[1] = {k.data, k.token_stride};
  a.dy[0] = {dqo.data, dqo.token_stride};
  a.dy[1] = {dko.data, dko.token_stride};
  a.y[0] = {dq.data, dq.token_stride};
  a.y[1] = {dk.data, dk.token_stride};
  a.dw[0] = dwq;
  a.dw[1] = dwk;
  return status_of(falcon::launch_qk_bwd(s->dtype == FALCON_BF16, s->grad_dtype == FALCON_F32, s->d, a, ws,
                                         static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- Causal attention ------------------------------------------------------------
namespace {

int64_t attn_tokens_q(const falcon_attn_shape_t *s, bool packed) {
  return packed ? s->seqlen_q : (int64_t)s->batch * s->seqlen_q;
}
int64_t attn_tokens_k(const falcon_attn_shape_t *s, bool packed) {
  return packed ? s->seqlen_k : (int64_t)s->batch * s->seqlen_k;
}

falcon::AttnArgs attn_args(const falcon_attn_shape_t *s, const int32_t *cu_q, const int32_t *cu_k) {
  falcon::AttnArgs a{};
  a.cuq = cu_q;
  a.cuk = cu_k;
  a.n = s->batch;
  a.Tq = s->seqlen_q;
  a.Tk = s->seqlen_k;
  a.hq = s->heads_q;
  a.hk = s->heads_k;
  a.group = s->heads_q / s->heads_k;
  a.scale = s->scale;
  return a;
}

// The fields that sizes depend on, for the workspace queries (any non-null offsets mark a packed call).
falcon::AttnArgs size_args(const falcon_attn_shape_t *s, bool packed) {
  static const int32_t mark = 0;
  return attn_args(s, packed ? &mark : nullptr, packed ? &mark : nullptr);
}

int check_attn(const falcon_attn_shape_t *s, bool packed) {
  if (!s || !dtype_ok(s->dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->batch < 1 || s->seqlen_q < 1 || s->seqlen_k < 1 || s->heads_q < 1 || s->heads_k < 1 || s->d < 1)
    return FALCON_ERR_INVALID_ARG;
  if (s->heads_q % s->heads_k != 0) return FALCON_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale) || !(s->scale > 0.f)) return FALCON_ERR_INVALID_ARG;
  FALCON_TRY(check_d(s->d));
  // token, row and sequence numbers are ints, with a tile added
  const int64_t tq = attn_tokens_q(s, packed), tk = attn_tokens_k(s, packed);
  if (tq > INT32_MAX - 4096 || tk > INT32_MAX - 4096 || s->heads_q > (1 << 20)) return FALCON_ERR_UNSUPPORTED;
  if (tq * (s->heads_q / s->heads_k) > INT32_MAX - 4096 || s->batch > (1 << 30)) return FALCON_ERR_UNSUPPORTED;
  return FALCON_OK;
}

// Of one direction: its launches too.
int check_attn_fwd(const falcon_attn_shape_t *s, bool packed) {
  FALCON_TRY(check_attn(s, packed));
  return falcon::attn_fwd_fits(s->dtype == FALCON_BF16, size_args(s, packed)) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}
int check_attn_bwd(const falcon_attn_shape_t *s, bool packed) {
  FALCON_TRY(check_attn(s, packed));
  return falcon::attn_bwd_fits(s->d, size_args(s, packed)) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}

constexpr int64_t MOST_STEP = 1 << 25;   // bytes between two tokens

int check_attn_in(const falcon_attn_shape_t *s, const int32_t *cu_q, const int32_t *cu_k, falcon_heads_t q,
                  falcon_heads_t k, falcon_heads_t v, const void *o) {
  if ((cu_q == nullptr) != (cu_k == nullptr)) return FALCON_ERR_INVALID_ARG;
  const bool packed = cu_q != nullptr;
  FALCON_TRY(check_attn(s, packed));
  FALCON_TRY(maybe(cu_q, 4));
  FALCON_TRY(maybe(cu_k, 4));
  const int e = esize(s->dtype);
  FALCON_TRY(check_heads(q.data, q.token_stride, attn_tokens_q(s, packed), s->heads_q, s->d, e));
  FALCON_TRY(check_heads(k.data, k.token_stride, attn_tokens_k(s, packed), s->heads_k, s->d, e));
  FALCON_TRY(check_heads(v.data, v.token_stride, attn_tokens_k(s, packed), s->heads_k, s->d, e));
  // the rows of a tile, at most 128, are 32 bits of bytes apart
  for (const int64_t stride : {q.token_stride, k.token_stride, v.token_stride})
    if (stride > MOST_STEP / e) return FALCON_ERR_UNSUPPORTED;
  return need(o, 16);
}

}  // namespace

extern "C" {

size_t falcon_attn_fwd_workspace(const falcon_attn_shape_t *s, int packed) {
  if (check_attn_fwd(s, packed != 0) != FALCON_OK) return 0;
  return falcon::attn_fwd_workspace(s->dtype == FALCON_BF16, s->d, size_args(s, packed != 0));
}

int falcon_attn_fwd(const falcon_attn_shape_t *s, const int32_t *cu_q, const int32_t *cu_k, falcon_heads_t q,
                    falcon_heads_t k, falcon_heads_t v, void *o, float *lse, void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_attn_in(s, cu_q, cu_k, q, k, v, o));
  FALCON_TRY(check_attn_fwd(s, cu_q != nullptr));
  FALCON_TRY(maybe(lse, 4));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_attn_fwd_workspace(s, cu_q != nullptr)));
  falcon::AttnArgs a = attn_args(s, cu_q, cu_k);
  a.q = q.data; a.k = k.data; a.v = v.data;
  a.ldq = q.token_stride; a.ldk = k.token_stride; a.ldv = v.token_stride;
  a.out = o;
  a.lse = lse;
  return status_of(falcon::launch_attn_fwd(s->dtype == FALCON_BF16, s->d, a, ws, static_cast<hipStream_t>(stream)));
}

size_t falcon_attn_bwd_workspace(const falcon_attn_shape_t *s, int packed) {
  if (check_attn_bwd(s, packed != 0) != FALCON_OK) return 0;
  return falcon::attn_bwd_workspace(s->d, size_args(s, packed != 0));
}

int falcon_attn_bwd(const falcon_attn_shape_t *s, const int32_t *cu_q, const int32_t *cu_k, falcon_heads_t q,
                    falcon_heads_t k, falcon_heads_t v, const void *o, const float *lse, falcon_heads_t d_o,
                    falcon_heads_out_t dq, falcon_heads_out_t dk, falcon_heads_out_t dv, void *ws, size_t ws_bytes,
                    void *stream) {
  FALCON_TRY(check_attn_in(s, cu_q, cu_k, q, k, v, o));
  const bool packed = cu_q != nullptr;
  FALCON_TRY(check_attn_bwd(s, packed));
  FALCON_TRY(need(lse, 4));
  const int64_t tq = attn_tokens_q(s, packed), tk = attn_tokens_k(s, packed);
  const int e = esize(s->dtype);
  FALCON_TRY(check_heads(d_o.data, d_o.token_stride, tq, s->heads_q, s->d, e));
  if (d_o.token_stride > MOST_STEP / e) return FALCON_ERR_UNSUPPORTED;
  FALCON_TRY(check_heads(dq.data, dq.token_stride, tq, s->heads_q, s->d, e));
  FALCON_TRY(check_heads(dk.data, dk.token_stride, tk, s->heads_k, s->d, e));
  FALCON_TRY(check_heads(dv.data, dv.token_stride, tk, s->heads_k, s->d, e));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_attn_bwd_workspace(s, packed)));
  falcon::AttnArgs a = attn_args(s, cu_q, cu_k);
  a.q = q.data; a.k = k.data; a.v = v.data;
  a.ldq = q.token_stride; a.ldk = k.token_stride; a.ldv = v.token_stride;
  a.o = o;
  a.lse_in = lse;
  a.d_o = d_o.data;
  a.lddo = d_o.token_stride;
  a.dq = dq.data; a.dk = dk.data; a.dv = dv.data;
  a.lddq = dq.token_stride; a.lddk = dk.token_stride; a.lddv = dv.token_stride;
  return status_of(falcon::launch_attn_bwd(s->dtype == FALCON_BF16, s->d, a, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
