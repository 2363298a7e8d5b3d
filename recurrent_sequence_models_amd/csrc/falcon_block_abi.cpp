// C ABI of the operators of a state-space block (declared in include/falcon.h): the norm of
// the residual stream, the short causal convolution, the selective state-space scan and the
// projections.
//
// Host side only, as falcon_layer_abi.cpp: every argument is validated before the first HIP
// call.
#include <iterator>

#include "abi_checks.h"
#include "block_kernels.h"

using namespace falcon::abi;

// ---- Norm of the residual stream -------------------------------------------------
namespace {

int check_norm(const falcon_norm_shape_t *s) {
  if (!s || !float_dtype(s->dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->tokens < 1 || s->width < 1 || (s->norm != 0 && s->norm != 1)) return FALCON_ERR_INVALID_ARG;
  if (!std::isfinite(s->eps) || s->eps < 0.f) return FALCON_ERR_INVALID_ARG;
  if (s->width % 8 != 0 || s->width > 65536 / esize(s->dtype)) return FALCON_ERR_UNSUPPORTED;
  return s->tokens > INT32_MAX - (1 << 20) ? FALCON_ERR_UNSUPPORTED : FALCON_OK;
}

falcon::NormArgs norm_args(const falcon_norm_shape_t *s, const float *w) {
  falcon::NormArgs a{};
  a.w = w;
  a.tokens = s->tokens;
  a.width = s->width;
  a.norm = s->norm;
  a.eps = s->eps;
  return a;
}

}  // namespace

extern "C" {

int falcon_rms_norm(const falcon_norm_shape_t *s, const void *x, const void *residual, const float *weight,
                    void *stream_out, void *y, float *scale, void *stream) {
  FALCON_TRY(check_norm(s));
  const bool q8 = s->out == FALCON_E4M3;
  if (!q8 && !float_dtype(s->out)) return FALCON_ERR_INVALID_ARG;
  if (!q8 && s->out != s->dtype) return FALCON_ERR_UNSUPPORTED;
  FALCON_TRY(need(x, 16));
  FALCON_TRY(maybe(residual, 16));
  FALCON_TRY(maybe(weight, 16));
  FALCON_TRY(maybe(stream_out, 16));
  FALCON_TRY(need(y, 16));
  FALCON_TRY(q8 ? need(scale, 4) : maybe(scale, 4));
  if (residual) FALCON_TRY(apart(stream_out, {weight, y}));
  FALCON_TRY(distinct(y, weight));
  if (q8) FALCON_TRY(apart(y, {x, residual}));                            // rows of another length
  if (q8) FALCON_TRY(apart(scale, {x, residual, weight, residual ? stream_out : nullptr, y}));
  falcon::NormArgs a = norm_args(s, weight);
  a.x = x;
  a.residual = residual;
  a.s = stream_out;
  a.y = y;
  a.scale = scale;
  return status_of(falcon::launch_norm_fwd(s->dtype == FALCON_BF16, q8, a, static_cast<hipStream_t>(stream)));
}

size_t falcon_rms_norm_bwd_workspace(const falcon_norm_shape_t *s) {
  if (check_norm(s) != FALCON_OK) return 0;
  return falcon::norm_bwd_workspace(s->dtype == FALCON_BF16, s->tokens, s->width);
}

int falcon_rms_norm_bwd(const falcon_norm_shape_t *s, const void *stream_in, const float *weight, const void *d_y,
                        const void *d_stream, void *dx, float *dweight, void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_norm(s));
  if (!s->norm) return FALCON_ERR_UNSUPPORTED;
  FALCON_TRY(need(stream_in, 16));
  FALCON_TRY(maybe(weight, 16));
  FALCON_TRY(need(d_y, 16));
  FALCON_TRY(maybe(d_stream, 16));
  FALCON_TRY(need(dx, 16));
  FALCON_TRY(maybe(dweight, 4));
  if (dweight) FALCON_TRY(check_workspace(ws, ws_bytes, falcon_rms_norm_bwd_workspace(s)));
  FALCON_TRY(apart(dx, {weight, dweight}));
  falcon::NormArgs a = norm_args(s, weight);
  a.x = stream_in;
  a.dy = d_y;
  a.ds = d_stream;
  a.y = dx;
  return status_of(falcon::launch_norm_bwd(s->dtype == FALCON_BF16, a, dweight, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- Short causal convolution ------------------------------------------------------
namespace {

int check_seq(int64_t batch, int64_t seqlen, bool packed) {
  if (batch < 1 || seqlen < 1) return FALCON_ERR_INVALID_ARG;
  // token and sequence numbers are ints, with a workgroup's tokens added
  if (batch > (1 << 30) || seqlen > INT32_MAX - 4096 || (!packed && batch * seqlen > INT32_MAX - 4096))
    return FALCON_ERR_UNSUPPORTED;
  return FALCON_OK;
}

falcon::SeqMap seq_map(int batch, int seqlen, const int32_t *cu) { return falcon::SeqMap{cu, batch, seqlen}; }

// The same for queries of sizes, where any non-null offsets mark a packed call.
falcon::SeqMap seq_sizes(int batch, int seqlen, bool packed) {
  static const int32_t mark = 0;
  return falcon::SeqMap{packed ? &mark : nullptr, batch, seqlen};
}

int check_conv(const falcon_conv_shape_t *s, bool packed, bool step) {
  if (!s || !float_dtype(s->dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->activation < FALCON_ACT_NONE || s->activation > FALCON_ACT_GELU) return FALCON_ERR_INVALID_ARG;
  if (s->width < 1 || s->taps < 1) return FALCON_ERR_INVALID_ARG;
  FALCON_TRY(check_seq(s->batch, step ? 1 : s->seqlen, packed));
  if (s->activation == FALCON_ACT_GELU || s->taps < 2 || s->taps > 4) return FALCON_ERR_UNSUPPORTED;
  if (s->width % 8 != 0 || s->width > (1 << 20)) return FALCON_ERR_UNSUPPORTED;
  const bool bf16 = s->dtype == FALCON_BF16;
  if (step) return falcon::conv_step_fits(bf16, s->batch, s->width) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
  return falcon::conv_fits(bf16, seq_sizes(s->batch, s->seqlen, packed), s->width) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}

falcon::ConvArgs conv_args(const falcon_conv_shape_t *s, const int32_t *cu, falcon_heads_t x, const float *w,
                           const float *bias) {
  falcon::ConvArgs a{};
  a.seq = seq_map(s->batch, s->seqlen, cu);
  a.x = x.data;
  a.ldx = x.token_stride;
  a.w = w;
  a.bias = bias;
  a.D = s->width;
  a.silu = s->activation == FALCON_ACT_SILU;
  return a;
}

int check_conv_in(const falcon_conv_shape_t *s, int64_t tokens, falcon_heads_t x, const float *w, const float *bias) {
  FALCON_TRY(check_rows(x.data, x.token_stride, tokens, s->width, esize(s->dtype)));
  FALCON_TRY(need(w, 4));
  return maybe(bias, 4);
}

int64_t seq_tokens(int64_t batch, int64_t seqlen, bool packed) { return packed ? seqlen : batch * seqlen; }

}  // namespace

extern "C" {

int falcon_conv_fwd(const falcon_conv_shape_t *s, const int32_t *cu, falcon_heads_t x, const float *w, const float *bias,
                    const void *init, void *final_state, void *y, void *stream) {
  FALCON_TRY(check_conv(s, cu != nullptr, false));
  FALCON_TRY(maybe(cu, 4));
  FALCON_TRY(check_conv_in(s, seq_tokens(s->batch, s->seqlen, cu), x, w, bias));
  FALCON_TRY(maybe(init, 16));
  FALCON_TRY(maybe(final_state, 16));
  FALCON_TRY(need(y, 16));
  FALCON_TRY(apart(final_state, {x.data, w, bias, init}));
  FALCON_TRY(apart(y, {x.data, w, bias, init, final_state}));
  falcon::ConvArgs a = conv_args(s, cu, x, w, bias);
  a.init = init;
  a.final_state = final_state;
  a.y = y;
  return status_of(falcon::launch_conv_fwd(s->dtype == FALCON_BF16, s->taps, a, static_cast<hipStream_t>(stream)));
}

size_t falcon_conv_bwd_workspace(const falcon_conv_shape_t *s, int packed) {
  if (check_conv(s, packed != 0, false) != FALCON_OK) return 0;
  return falcon::conv_bwd_workspace(s->dtype == FALCON_BF16, s->taps, seq_sizes(s->batch, s->seqlen, packed != 0), s->width);
}

int falcon_conv_bwd(const falcon_conv_shape_t *s, const int32_t *cu, falcon_heads_t x, const float *w, const float *bias,
                    const void *init, const void *d_y, const void *d_final, falcon_heads_out_t dx, float *dw, float *db,
                    void *d_init, void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_conv(s, cu != nullptr, false));
  FALCON_TRY(maybe(cu, 4));
  const int64_t tokens = seq_tokens(s->batch, s->seqlen, cu);
  FALCON_TRY(check_conv_in(s, tokens, x, w, bias));
  FALCON_TRY(maybe(init, 16));
  FALCON_TRY(need(d_y, 16));
  FALCON_TRY(maybe(d_final, 16));
  FALCON_TRY(check_rows(dx.data, dx.token_stride, tokens, s->width, esize(s->dtype)));
  FALCON_TRY(maybe(dw, 4));
  FALCON_TRY(maybe(db, 4));
  FALCON_TRY(maybe(d_init, 16));
  if (dw || db) FALCON_TRY(check_workspace(ws, ws_bytes, falcon_conv_bwd_workspace(s, cu != nullptr)));
  // d_init too: runs behind a sequence's first one may read the inputs before it still
  for (const void *out : {(const void *)dx.data, (const void *)d_init})
    FALCON_TRY(apart(out, {x.data, w, bias, init, d_y, d_final, dw, db}));
  FALCON_TRY(distinct(dx.data, d_init));
  FALCON_TRY(distinct(dw, db));
  falcon::ConvArgs a = conv_args(s, cu, x, w, bias);
  a.init = init;
  a.dy = d_y;
  a.d_final = d_final;
  a.dx = dx.data;
  a.lddx = dx.token_stride;
  a.d_init = d_init;
  return status_of(falcon::launch_conv_bwd(s->dtype == FALCON_BF16, s->taps, a, dw, db, ws,
                                           static_cast<hipStream_t>(stream)));
}

int falcon_conv_step(const falcon_conv_shape_t *s, falcon_heads_t x, const float *w, const float *bias, const void *state,
                     void *state_out, void *y, void *stream) {
  FALCON_TRY(check_conv(s, false, true));
  FALCON_TRY(check_conv_in(s, s->batch, x, w, bias));
  FALCON_TRY(need(state, 16));
  FALCON_TRY(need(state_out, 16));
  FALCON_TRY(need(y, 16));
  FALCON_TRY(apart(y, {w, bias, state, state_out}));
  FALCON_TRY(apart(state_out, {x.data, w, bias}));
  FALCON_TRY(same_rows(y, s->width, x.data, x.token_stride, s->batch));
  falcon::ConvArgs a = conv_args(s, nullptr, x, w, bias);
  a.init = state;
  a.final_state = state_out;
  a.y = y;
  return status_of(falcon::launch_conv_step(s->dtype == FALCON_BF16, s->taps, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- Selective state-space scan ------------------------------------------------------
namespace {

int check_ssm(const falcon_ssm_shape_t *s, bool packed, bool step) {
  if (!s || !float_dtype(s->dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->width < 1 || s->state < 1 || (s->softplus != 0 && s->softplus != 1)) return FALCON_ERR_INVALID_ARG;
  FALCON_TRY(check_seq(s->batch, step ? 1 : s->seqlen, packed));
  if (s->state != 16 && s->state != 32 && s->state != 64) return FALCON_ERR_UNSUPPORTED;
  if (s->width % 8 != 0 || s->width > (1 << 20)) return FALCON_ERR_UNSUPPORTED;
  if (step) return falcon::ssm_step_fits(s->batch, s->width, s->state) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
  return falcon::ssm_fits(seq_sizes(s->batch, s->seqlen, packed), s->width, s->state) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}

// [tokens, width] whose tokens are at most 2^24 bytes apart: the rows of a tile, at most 64, are 32 bits apart.
int check_near(const void *p, int64_t stride, int64_t tokens, int64_t width, int e) {
  FALCON_TRY(check_rows(p, stride, tokens, width, e));
  return stride > (1 << 24) / e ? FALCON_ERR_UNSUPPORTED : FALCON_OK;
}

int check_ssm_in(const falcon_ssm_shape_t *s, int64_t tokens, falcon_heads_t x, falcon_heads_t dt, const float *A,
                 falcon_heads_t B, falcon_heads_t C, const float *D, falcon_heads_t z, const float *bias) {
  const int e = esize(s->dtype);
  FALCON_TRY(check_near(x.data, x.token_stride, tokens, s->width, e));
  FALCON_TRY(check_near(dt.data, dt.token_stride, tokens, s->width, e));
  FALCON_TRY(need(A, 16));
  FALCON_TRY(check_near(B.data, B.token_stride, tokens, s->state, e));
  FALCON_TRY(check_near(C.data, C.token_stride, tokens, s->state, e));
  FALCON_TRY(maybe(D, 4));
  if (z.data) FALCON_TRY(check_near(z.data, z.token_stride, tokens, s->width, e));
  return maybe(bias, 4);
}

falcon::SsmArgs ssm_args(const falcon_ssm_shape_t *s, const int32_t *cu, falcon_heads_t x, falcon_heads_t dt,
                         const float *A, falcon_heads_t B, falcon_heads_t C, const float *D, falcon_heads_t z,
                         const float *bias) {
  falcon::SsmArgs a{};
  a.seq = seq_map(s->batch, s->seqlen, cu);
  a.x = x.data; a.dt = dt.data; a.z = z.data; a.B = B.data; a.C = C.data;
  a.ldx = x.token_stride; a.lddt = dt.token_stride; a.ldz = z.token_stride;
  a.ldB = B.token_stride; a.ldC = C.token_stride;
  a.A = A;
  a.skip = D;
  a.bias = bias;
  a.D = s->width;
  a.softplus = s->softplus;
  return a;
}

}  // namespace

extern "C" {

size_t falcon_ssm_fwd_workspace(const falcon_ssm_shape_t *s, int packed) {
  if (check_ssm(s, packed != 0, false) != FALCON_OK) return 0;
  return falcon::ssm_fwd_workspace(seq_sizes(s->batch, s->seqlen, packed != 0), s->width, s->state);
}

int falcon_ssm_chunks(const falcon_ssm_shape_t *s, int packed) {
  if (check_ssm(s, packed != 0, false) != FALCON_OK) return 0;
  const int K = falcon::ssm_chunk(s->state);
  if (packed) return s->seqlen / K + s->batch;
  return s->batch * ((s->seqlen + K - 1) / K);
}

int falcon_ssm_fwd(const falcon_ssm_shape_t *s, const int32_t *cu, falcon_heads_t x, falcon_heads_t dt, const float *A,
                   falcon_heads_t B, falcon_heads_t C, const float *D, falcon_heads_t z, const float *bias,
                   const float *init, float *final_state, void *y, float *chunk_states, void *ws, size_t ws_bytes,
                   void *stream) {
  FALCON_TRY(check_ssm(s, cu != nullptr, false));
  FALCON_TRY(maybe(cu, 4));
  FALCON_TRY(check_ssm_in(s, seq_tokens(s->batch, s->seqlen, cu), x, dt, A, B, C, D, z, bias));
  FALCON_TRY(maybe(init, 16));
  FALCON_TRY(maybe(final_state, 16));
  FALCON_TRY(need(y, 16));
  FALCON_TRY(maybe(chunk_states, 16));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_ssm_fwd_workspace(s, cu != nullptr)));
  FALCON_TRY(apart(y, {A, B.data, C.data, D, bias, init, final_state, chunk_states}));
  FALCON_TRY(apart(final_state, {x.data, dt.data, A, B.data, C.data, D, z.data, bias, init, chunk_states}));
  FALCON_TRY(apart(chunk_states, {x.data, dt.data, A, B.data, C.data, D, z.data, bias, init}));
  for (const falcon_heads_t &t : {x, dt, z})
    FALCON_TRY(same_rows(y, s->width, t.data, t.token_stride, seq_tokens(s->batch, s->seqlen, cu)));
  falcon::SsmArgs a = ssm_args(s, cu, x, dt, A, B, C, D, z, bias);
  a.init = init;
  a.final_state = final_state;
  a.y = y;
  a.states = chunk_states;
  return status_of(falcon::launch_ssm_fwd(s->dtype == FALCON_BF16, s->state, a, ws, static_cast<hipStream_t>(stream)));
}

// Of the backward: its launches for the sums over workgroups too.
static int check_ssm_bwd(const falcon_ssm_shape_t *s, bool packed) {
  FALCON_TRY(check_ssm(s, packed, false));
  const int64_t sums = seq_tokens(s->batch, s->seqlen, packed) * s->state / 2;
  return falcon::grid_fits((sums + 255) / 256, 256) && falcon::grid_fits((int64_t)s->width * s->state / 16, 1024)
             ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}

size_t falcon_ssm_bwd_workspace(const falcon_ssm_shape_t *s, int packed) {
  if (check_ssm_bwd(s, packed != 0) != FALCON_OK) return 0;
  return falcon::ssm_bwd_workspace(seq_sizes(s->batch, s->seqlen, packed != 0), s->width, s->state);
}

int falcon_ssm_bwd(const falcon_ssm_shape_t *s, const int32_t *cu, falcon_heads_t x, falcon_heads_t dt, const float *A,
                   falcon_heads_t B, falcon_heads_t C, const float *D, falcon_heads_t z, const float *bias,
                   const float *chunk_states, const void *d_y, const float *d_final, falcon_heads_out_t dx,
                   falcon_heads_out_t ddt, float *dA, falcon_heads_out_t dB, falcon_heads_out_t dC, float *dD,
                   falcon_heads_out_t dz, float *ddt_bias, float *d_init, void *ws, size_t ws_bytes, void *stream) {
  FALCON_TRY(check_ssm_bwd(s, cu != nullptr));
  FALCON_TRY(maybe(cu, 4));
  const int64_t tokens = seq_tokens(s->batch, s->seqlen, cu);
  FALCON_TRY(check_ssm_in(s, tokens, x, dt, A, B, C, D, z, bias));
  FALCON_TRY(need(chunk_states, 16));
  FALCON_TRY(need(d_y, 16));
  FALCON_TRY(maybe(d_final, 16));
  const int e = esize(s->dtype);
  FALCON_TRY(check_near(dx.data, dx.token_stride, tokens, s->width, e));
  FALCON_TRY(check_near(ddt.data, ddt.token_stride, tokens, s->width, e));
  FALCON_TRY(check_near(dB.data, dB.token_stride, tokens, s->state, e));
  FALCON_TRY(check_near(dC.data, dC.token_stride, tokens, s->state, e));
  if (z.data) FALCON_TRY(check_near(dz.data, dz.token_stride, tokens, s->width, e));
  FALCON_TRY(need(dA, 4));
  FALCON_TRY(maybe(dD, 4));
  FALCON_TRY(maybe(ddt_bias, 4));
  FALCON_TRY(maybe(d_init, 16));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_ssm_bwd_workspace(s, cu != nullptr)));
  // A pass over the sequences writes dx, ddt, dz and d_init; those behind it, which read no inputs, the rest.
  FALCON_TRY(apart(d_init, {x.data, dt.data, A, B.data, C.data, D, z.data, bias, chunk_states, d_y, d_final}));
  const falcon_heads_out_t rows[] = {dx, ddt, z.data ? dz : falcon_heads_out_t{}};
  for (const falcon_heads_out_t &o : rows) {
    FALCON_TRY(apart(o.data, {A, B.data, C.data, D, bias, chunk_states, d_final}));
    for (const falcon_heads_t &t : {x, dt, z}) FALCON_TRY(same_rows(o.data, o.token_stride, t.data, t.token_stride, tokens));
    FALCON_TRY(same_rows(o.data, o.token_stride, d_y, s->width, tokens));
  }
  const void *outs[] = {dx.data, ddt.data, rows[2].data, dB.data, dC.data, dA, dD, ddt_bias, d_init};
  for (const void **o = outs; o != std::end(outs); ++o)
    for (const void **p = outs; p != o; ++p) FALCON_TRY(distinct(*o, *p));
  falcon::SsmArgs a = ssm_args(s, cu, x, dt, A, B, C, D, z, bias);
  a.states = const_cast<float *>(chunk_states);
  a.dy = d_y;
  a.d_final = d_final;
  a.dx = dx.data; a.ddt = ddt.data; a.dz = dz.data; a.dB = dB.data; a.dC = dC.data;
  a.lddx = dx.token_stride; a.ldddt = ddt.token_stride; a.lddz = dz.token_stride;
  a.lddB = dB.token_stride; a.lddC = dC.token_stride;
  a.d_init = d_init;
  return status_of(falcon::launch_ssm_bwd(s->dtype == FALCON_BF16, s->state, a, falcon::SsmGrads{dA, dD, ddt_bias}, ws,
                                          static_cast<hipStream_t>(stream)));
}

int falcon_ssm_step(const falcon_ssm_shape_t *s, falcon_heads_t x, falcon_heads_t dt, const float *A, falcon_heads_t B,
                    falcon_heads_t C, const float *D, falcon_heads_t z, const float *bias, const float *state,
                    float *state_out, void *y, void *stream) {
  FALCON_TRY(check_ssm(s, false, true));
  FALCON_TRY(check_ssm_in(s, s->batch, x, dt, A, B, C, D, z, bias));
  FALCON_TRY(need(state, 16));
  FALCON_TRY(need(state_out, 16));
  FALCON_TRY(need(y, 16));
  FALCON_TRY(apart(y, {A, B.data, C.data, D, bias, state, state_out}));
  FALCON_TRY(apart(state_out, {x.data, dt.data, A, B.data, C.data, D, z.data, bias}));
  for (const falcon_heads_t &t : {x, dt, z}) FALCON_TRY(same_rows(y, s->width, t.data, t.token_stride, s->batch));
  falcon::SsmArgs a = ssm_args(s, nullptr, x, dt, A, B, C, D, z, bias);
  a.seq.T = 1;
  a.init = state;
  a.final_state = state_out;
  a.y = y;
  return status_of(falcon::launch_ssm_step(s->dtype == FALCON_BF16, s->state, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- Projections -----------------------------------------------------------------------
namespace {

int check_linear(const falcon_linear_shape_t *s) {
  if (!s || (!float_dtype(s->dtype) && s->dtype != FALCON_E4M3) || !float_dtype(s->out_dtype)) return FALCON_ERR_INVALID_ARG;
  if (s->activation < FALCON_ACT_NONE || s->activation > FALCON_ACT_GELU) return FALCON_ERR_INVALID_ARG;
  if (s->tokens < 1 || s->in < 1 || s->out < 1) return FALCON_ERR_INVALID_ARG;
  if (s->dtype != FALCON_E4M3 && s->out_dtype != s->dtype) return FALCON_ERR_UNSUPPORTED;
  if (s->in % 16 != 0 || s->out % 8 != 0 || s->in > (1 << 20) || s->out > (1 << 20)) return FALCON_ERR_UNSUPPORTED;
  // token numbers are ints, with a tile added
  if (s->tokens > INT32_MAX - 4096) return FALCON_ERR_UNSUPPORTED;
  return falcon::linear_fits(esize(s->dtype), s->tokens, s->in, s->out) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}

constexpr int64_t MOST_STEP = 1 << 23;   // bytes between two tokens: the rows of a tile, at most 256, are 32 bits apart

int check_operand(falcon_heads_t t, int64_t tokens, int64_t width, int e) {
  FALCON_TRY(check_rows(t.data, t.token_stride, tokens, width, e));
  return t.token_stride > MOST_STEP / e ? FALCON_ERR_UNSUPPORTED : FALCON_OK;
}

}  // namespace

extern "C" {

size_t falcon_linear_fwd_workspace(const falcon_linear_shape_t *s) {
  if (check_linear(s) != FALCON_OK) return 0;
  return falcon::linear_fwd_workspace(esize(s->dtype), s->tokens, s->in, s->out);
}

int falcon_linear_fwd(const falcon_linear_shape_t *s, falcon_heads_t x, const void *weight, const float *x_scale,
                      const float *weight_scale, const float *bias, const void *residual, void *y, float *pre, void *ws,
                      size_t ws_bytes, void *stream) {
  FALCON_TRY(check_linear(s));
  FALCON_TRY(check_operand(x, s->tokens, s->in, esize(s->dtype)));
  FALCON_TRY(need(weight, 16));
  const bool q8 = s->dtype == FALCON_E4M3;
  if (q8 ? !x_scale || !weight_scale : x_scale || weight_scale) return FALCON_ERR_INVALID_ARG;
  FALCON_TRY(maybe(x_scale, 4));
  FALCON_TRY(maybe(weight_scale, 4));
  FALCON_TRY(maybe(bias, 4));
  FALCON_TRY(maybe(residual, 16));
  FALCON_TRY(need(y, 16));
  FALCON_TRY(maybe(pre, 16));
  FALCON_TRY(distinct(y, pre));
  FALCON_TRY(distinct(pre, residual));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_linear_fwd_workspace(s)));
  // Workgroups store while others copy operands.  One token's bias and scales of W are read by the threads that store there.
  for (const void *out : {(const void *)y, (const void *)pre}) {
    FALCON_TRY(apart(out, {x.data, weight, x_scale}));
    if (s->tokens > 1) FALCON_TRY(apart(out, {weight_scale, bias}));
  }
  falcon::LinearArgs a{};
  a.left = weight; a.ldl = s->in;
  a.right = x.data; a.ldr = x.token_stride;
  a.I = s->out; a.J = s->tokens; a.K = s->in;
  a.out = y; a.ldo = s->out;
  a.pre = pre;
  a.scale_l = weight_scale; a.scale_r = x_scale;
  a.bias = bias;
  a.residual = residual;
  a.act = s->activation;
  return status_of(falcon::launch_linear_fwd(s->dtype, s->out_dtype == FALCON_BF16, a, ws, static_cast<hipStream_t>(stream)));
}

size_t falcon_linear_bwd_workspace(const falcon_linear_shape_t *s) {
  if (check_linear(s) != FALCON_OK || s->dtype == FALCON_E4M3) return 0;
  return falcon::linear_bwd_workspace(esize(s->dtype), s->activation != FALCON_ACT_NONE, s->tokens, s->in, s->out);
}

int falcon_linear_bwd(const falcon_linear_shape_t *s, falcon_heads_t x, const void *weight, const float *pre,
                      falcon_heads_t d_y, falcon_heads_out_t dx, void *dweight, float *dbias, void *ws, size_t ws_bytes,
                      void *stream) {
  FALCON_TRY(check_linear(s));
  if (s->dtype == FALCON_E4M3) return FALCON_ERR_UNSUPPORTED;
  const int e = esize(s->dtype);
  const bool act = s->activation != FALCON_ACT_NONE;
  if (dweight) FALCON_TRY(check_operand(x, s->tokens, s->in, e));
  if (dx.data) FALCON_TRY(need(weight, 16));
  FALCON_TRY(act ? need(pre, 16) : FALCON_OK);
  FALCON_TRY(check_operand(d_y, s->tokens, s->out, e));
  if (dx.data) FALCON_TRY(check_rows(dx.data, dx.token_stride, s->tokens, s->in, e));
  FALCON_TRY(maybe(dweight, 16));
  FALCON_TRY(maybe(dbias, 4));
  FALCON_TRY(distinct(dx.data, d_y.data));
  FALCON_TRY(distinct(dx.data, x.data));
  FALCON_TRY(distinct(dweight, weight));
  FALCON_TRY(check_workspace(ws, ws_bytes, falcon_linear_bwd_workspace(s)));
  // dbias, dx and dweight are written in this order; a product copies its operands while others' tiles are stored
  FALCON_TRY(distinct(dx.data, weight));
  FALCON_TRY(apart(dweight, {x.data, d_y.data, dx.data}));
  FALCON_TRY(apart(dbias, {x.data, d_y.data, weight, dx.data, dweight}));
  falcon::LinearGrads g{};
  g.x = x.data; g.ldx = x.token_stride;
  g.w = weight;
  g.pre = pre;
  g.dy = d_y.data; g.lddy = d_y.token_stride;
  g.dx = dx.data; g.lddx = dx.token_stride;
  g.dw = dweight;
  g.dbias = dbias;
  g.tokens = s->tokens; g.in = s->in; g.out = s->out;
  g.act = s->activation;
  return status_of(falcon::launch_linear_bwd(s->dtype == FALCON_BF16, g, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
