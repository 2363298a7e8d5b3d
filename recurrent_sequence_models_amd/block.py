"""Python binding of the operators of a state-space block (include/falcon.h): the norm of
the residual stream with its output in 8 bits, the projections with their epilogues, the
short causal convolution, and the selective state-space scan.

Argument marshalling only, as layer.py, whose conventions of devices, streams and
workspaces hold here.  A tensor given for an output is none of the inputs or other outputs,
unless the function's text says so (FALCON_ERR_INVALID_ARG where it would be a race).
"""

from __future__ import annotations

import ctypes
import functools

from .falcon import ConvShape, Heads, LinearShape, NormShape, SsmShape, lib
from .layer import _check, _current, _device, _done, _dtype, _ints, _offsets, _on, _p, _types, _workspace

E4M3 = 2   # FALCON_E4M3
ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2}


@functools.lru_cache(maxsize=None)
def _f8():
    import torch
    return torch.float8_e4m3fn


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation: {name!r}, expected None, 'silu' or 'gelu'")
    return ACTIVATIONS[name]


def _rows(name, t, dtype, dev, shape=None):
    """falcon_heads_t of t [..., width] (of this shape, if given): dense rows, tokens one
    stride apart (views of a wider projection are taken as they are)."""
    size = t.shape
    if t.is_contiguous() and t.dtype is dtype and (shape is None or size == shape) and t.device == dev:
        return Heads(t.data_ptr(), size[-1])
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and size != shape:
        raise ValueError(f"{name}: shape {tuple(size)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: must live on {dev}")
    step = size[-1]
    *strides, sd = t.stride()
    want, ok = None, sd == 1 or size[-1] == 1
    for n, s in zip(reversed(size[:-1]), reversed(strides)):
        if n == 1:
            continue
        if want is None:
            step = want = s
        ok = ok and s == want
        want = want * n
    if not ok or step < size[-1]:
        raise ValueError(f"{name}: rows must be dense and tokens one stride apart")
    if (step * t.element_size()) % 16:
        raise ValueError(f"{name}: the distance of two tokens must be a multiple of 16 bytes")
    return Heads(t.data_ptr(), step)


def _like(x):
    """A new dense tensor of x's type and shape (by the quick way where x is dense)."""
    import torch
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(tuple(x.shape))


def _maybe(name, t, dtype, shape, dev):
    if t is not None:
        _check(name, t, dtype, shape, dev)
    return t


# ---- Norm of the residual stream ----------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _norm_plan(dtype, tokens, width, norm, out, eps):
    """(pointer to the C shape, workspace bytes of the backward)."""
    shape = NormShape(dtype, *_ints(tokens, width), norm, out, eps)
    return ctypes.pointer(shape), lib().falcon_rms_norm_bwd_workspace(ctypes.byref(shape))


def _norm_shape(name, x, norm, out, eps):
    dt, dev = _dtype(name, x), _device(name, x)
    if x.dim() < 1:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected [..., width]")
    _check(name, x, x.dtype, x.shape, dev)
    width = x.shape[-1]
    plan = _norm_plan(dt, x.numel() // max(width, 1), width, norm, dt if out is None else out, float(eps))
    return *plan, width, dev


def _norm_fwd(x, weight, residual, norm, eps, quantize, out, scale, stream_out, stream):
    import torch
    shape, _, width, dev = _norm_shape("x", x, norm, E4M3 if quantize else None, eps)
    _maybe("weight", weight, torch.float32, (width,), dev)
    _maybe("residual", residual, x.dtype, x.shape, dev)
    if stream_out is not None and residual is None:
        raise ValueError("stream_out: the stream is x itself without a residual")
    with _on(dev, stream):
        ydt = _f8() if quantize else x.dtype
        if out is None:
            out = torch.empty_like(x, dtype=ydt)
        else:
            _check("y", out, ydt, x.shape, dev)
        if residual is None:
            stream_out = None
        elif stream_out is None:
            stream_out = torch.empty_like(x)
        else:
            _check("stream_out", stream_out, x.dtype, x.shape, dev)
        if not quantize:
            scale = None
        elif scale is None:
            scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
        else:
            _check("scale", scale, torch.float32, x.shape[:-1], dev)
        _done(lib().falcon_rms_norm(shape, _p(x), _p(residual), _p(weight), _p(stream_out), _p(out), _p(scale),
                                    _current(dev)), "falcon_rms_norm")
    return out, x if residual is None else stream_out, scale


def rms_norm(x, weight, *, residual=None, eps=1e-6, quantize=False, out=None, scale=None, stream_out=None, stream=None):
    """falcon_rms_norm on torch tensors: the norm of the residual stream s = x + residual,
    y = s weight / sqrt(mean(s^2) + eps) over the last axis.

    x, residual [..., width] (float32 or bfloat16, width a multiple of 8), weight [width]
    float32 or None (ones).  s is rounded to the inputs' type; the norm is of the rounded
    sum.  ``quantize``: y as float8_e4m3fn with one float32 scale a token (what ``linear``
    takes as x and x_scale).  ``out``, ``scale``, ``stream_out``: None or preallocated;
    stream_out may be residual or x.  Returns (y, s, scale): s is x itself without a
    residual, scale None without ``quantize``."""
    return _norm_fwd(x, weight, residual, 1, eps, quantize, out, scale, stream_out, stream)


def quantize_rows(x, *, out=None, scale=None, stream=None):
    """falcon_rms_norm without its norm: the rows of x [..., width] (float32 or bfloat16)
    as float8_e4m3fn with one float32 scale a row, x ~ q scale.  For ``linear``'s weights,
    and activations that no norm precedes.  Returns (q, scale)."""
    q, _, scale = _norm_fwd(x, None, None, 0, 0.0, True, out, scale, None, stream)
    return q, scale


def rms_norm_bwd(s, weight, dy, *, d_stream=None, eps=1e-6, dweight=True, out=None, workspace=None, stream=None):
    """falcon_rms_norm_bwd on torch tensors: gradients of <dy, y> + <d_stream, s> for
    ``rms_norm`` of the same weight and eps, which gave the stream s.

    dy, d_stream (or None) have the dtype and shape of s.  ``dweight``: whether to return
    the weight's gradient.  ``out``: None or a tensor for dx (dy or d_stream will do).
    Returns dict(dx, dweight): dx is the gradient of x and of the residual alike; dweight
    [width] float32 (None without a weight)."""
    import torch
    shape, need, width, dev = _norm_shape("s", s, 1, None, eps)
    _maybe("weight", weight, torch.float32, (width,), dev)
    _check("dy", dy, s.dtype, s.shape, dev)
    _maybe("d_stream", d_stream, s.dtype, s.shape, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(s)
        else:
            _check("dx", out, s.dtype, s.shape, dev)
        dw = s.new_empty((width,), dtype=torch.float32) if dweight and weight is not None else None
        ws, nbytes = _workspace(need if dw is not None else 0, workspace, dev)
        _done(lib().falcon_rms_norm_bwd(shape, _p(s), _p(weight), _p(dy), _p(d_stream), _p(out), _p(dw), _p(ws), nbytes,
                                        _current(dev)), "falcon_rms_norm_bwd")
    return dict(dx=out, dweight=dw)


# ---- Sequences ------------------------------------------------------------------------

def _sequences(x, cu_seqlens):
    """(sequences, tokens of one or of all) of x [B, T, D], or [total, D] with offsets."""
    if x.dim() != (3 if cu_seqlens is None else 2):
        raise ValueError(f"x: shape {tuple(x.shape)}, expected " + ("[B, T, D]" if cu_seqlens is None else "[total, D]"))
    if cu_seqlens is None:
        return x.shape[0], x.shape[1]
    return _offsets("cu_seqlens", cu_seqlens, x.device), x.shape[0]


# ---- Short causal convolution -----------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _conv_plan(dtype, n, T, D, taps, act, packed):
    """(pointer to the C shape, workspace bytes of the backward)."""
    shape = ConvShape(dtype, *_ints(n, T, D, taps), act)
    return ctypes.pointer(shape), lib().falcon_conv_bwd_workspace(ctypes.byref(shape), packed)


def _conv_shape(x, weight, bias, activation, cu_seqlens):
    import torch
    dt, dev = _dtype("x", x), _device("x", x)
    n, T = _sequences(x, cu_seqlens)
    D = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected [D, taps]")
    taps = weight.shape[1]
    _check("weight", weight, torch.float32, (D, taps), dev)
    _maybe("bias", bias, torch.float32, (D,), dev)
    hx = _rows("x", x, x.dtype, dev)
    return *_conv_plan(dt, n, T, D, taps, _activation(activation), cu_seqlens is not None), hx, (n, taps - 1, D), dev


def causal_conv(x, weight, *, bias=None, activation=None, cu_seqlens=None, init=None, final=True, out=None, stream=None):
    """falcon_conv_fwd on torch tensors: y_t = act(bias + sum_j weight_j x_{t-taps+1+j})
    per channel.

    x [B,T,D] (float32 or bfloat16, D a multiple of 8; a view of a wider projection will
    do), or [total,D] with ``cu_seqlens``, an int32 device tensor [N+1] of token offsets;
    weight [D,taps] float32 with 2 to 4 taps, bias [D] float32; ``activation``: None or
    "silu".  ``init``: None or [N,taps-1,D] in the dtype of x, the inputs before each
    sequence, oldest first.  ``final``: True (allocate), such a tensor to write, or False.
    Tokens behind cu_seqlens[N] are not written.  Returns (y, final)."""
    import torch
    shape, _, hx, states, dev = _conv_shape(x, weight, bias, activation, cu_seqlens)
    _maybe("init", init, x.dtype, states, dev)
    with _on(dev, stream):
        if out is None:
            out = _like(x)
        else:
            _check("y", out, x.dtype, x.shape, dev)
        final = x.new_empty(states) if final is True else None if final is False else final
        _maybe("final", final, x.dtype, states, dev)
        _done(lib().falcon_conv_fwd(shape, _p(cu_seqlens), hx, _p(weight), _p(bias), _p(init), _p(final), _p(out),
                                    _current(dev)), "falcon_conv_fwd")
    return out, final


def causal_conv_bwd(x, weight, dy, *, bias=None, activation=None, cu_seqlens=None, init=None, d_final=None, d_init=True,
                    out=None, workspace=None, stream=None):
    """falcon_conv_bwd on torch tensors: gradients of <dy, y> + <d_final, final> for
    ``causal_conv`` of the same arguments.

    dy has the dtype and shape of x, d_final (or None) those of its final state.
    ``d_init``: True (allocate), a tensor like init, or False.  ``out``: None or a tensor
    for dx (a view with dense rows will do).  Returns dict(dx, dweight, dbias, d_init):
    dweight [D,taps] and dbias [D] float32 (dbias None without a bias)."""
    import torch
    shape, need, hx, states, dev = _conv_shape(x, weight, bias, activation, cu_seqlens)
    _maybe("init", init, x.dtype, states, dev)
    _check("dy", dy, x.dtype, x.shape, dev)
    _maybe("d_final", d_final, x.dtype, states, dev)
    with _on(dev, stream):
        if out is None:
            out = _like(x)
        hdx = _rows("dx", out, x.dtype, dev, x.shape)
        d_init = x.new_empty(states) if d_init is True else None if d_init is False else d_init
        _maybe("d_init", d_init, x.dtype, states, dev)
        dw = torch.empty_like(weight)
        db = torch.empty_like(bias) if bias is not None else None
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_conv_bwd(shape, _p(cu_seqlens), hx, _p(weight), _p(bias), _p(init), _p(dy), _p(d_final), hdx,
                                    _p(dw), _p(db), _p(d_init), _p(ws), nbytes, _current(dev)), "falcon_conv_bwd")
    return dict(dx=out, dweight=dw, dbias=db, d_init=d_init)


def causal_conv_step(x, weight, state, *, bias=None, activation=None, state_out=None, out=None, stream=None):
    """falcon_conv_step: one token of every sequence; x [B,D], ``state`` [B,taps-1,D] in
    the dtype of x, updated in place, or left as it is with ``state_out``, a tensor for
    the new state.  Returns y [B,D]."""
    import torch
    dt, dev = _dtype("x", x), _device("x", x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"x, weight: shapes {tuple(x.shape)}, {tuple(weight.shape)}, expected [B, D], [D, taps]")
    (B, D), taps = x.shape, weight.shape[1]
    _check("weight", weight, torch.float32, (D, taps), dev)
    _maybe("bias", bias, torch.float32, (D,), dev)
    hx = _rows("x", x, x.dtype, dev)
    if state_out is None:
        state_out = state
    for name, t in (("state", state), ("state_out", state_out)):
        _check(name, t, x.dtype, (B, taps - 1, D), dev)
    with _on(dev, stream):
        if out is None:
            out = _like(x)
        else:
            _check("y", out, x.dtype, x.shape, dev)
        shape, _ = _conv_plan(dt, B, 1, D, taps, _activation(activation), False)
        _done(lib().falcon_conv_step(shape, hx, _p(weight), _p(bias), _p(state), _p(state_out), _p(out), _current(dev)),
              "falcon_conv_step")
    return out


# ---- Selective state-space scan ------------------------------------------------------------

_NO_ROWS = Heads(None, 0)


@functools.lru_cache(maxsize=1024)
def _ssm_plan(dtype, n, T, D, N, softplus, packed):
    """(pointer to the C shape, chunks, workspace bytes of the forward, of the backward)."""
    shape = SsmShape(dtype, *_ints(n, T, D, N), softplus)
    L, ref = lib(), ctypes.byref(shape)
    return (ctypes.pointer(shape), L.falcon_ssm_chunks(ref, packed), L.falcon_ssm_fwd_workspace(ref, packed),
            L.falcon_ssm_bwd_workspace(ref, packed))


def _ssm_args(x, dt, A, B, C, D, z, dt_bias):
    """The checked arguments as the C calls take them, (x, dt, A, B, C, D, z, dt_bias)."""
    import torch
    dev, lead, width = x.device, x.shape[:-1], x.shape[-1]
    if A.dim() != 2:
        raise ValueError(f"A: shape {tuple(A.shape)}, expected [D, N]")
    N = A.shape[1]
    _check("A", A, torch.float32, (width, N), dev)
    _maybe("D", D, torch.float32, (width,), dev)
    _maybe("dt_bias", dt_bias, torch.float32, (width,), dev)
    kind, states = x.dtype, lead + (N,)
    return (_rows("x", x, kind, dev), _rows("dt", dt, kind, dev, x.shape), _p(A), _rows("B", B, kind, dev, states),
            _rows("C", C, kind, dev, states), _p(D), _NO_ROWS if z is None else _rows("z", z, kind, dev, x.shape), _p(dt_bias))


def selective_scan(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, cu_seqlens=None, init=None, final=True,
                   chunk_states=False, out=None, workspace=None, stream=None):
    """falcon_ssm_fwd on torch tensors: per channel d and state n, with delta =
    softplus(dt + dt_bias) (or dt + dt_bias without ``softplus``),
    h_t = exp(delta_t A[d,n]) h_{t-1} + delta_t x_t B_t[n] and
    y_t = (sum_n C_t[n] h_t + D[d] x_t) silu(z_t).

    x, dt, z [B,T,D] and B, C [B,T,N] (float32 or bfloat16, D a multiple of 8, N 16, 32 or
    64; views of a wider projection will do), or [total,...] with ``cu_seqlens``, an int32
    device tensor [N+1] of token offsets.  A [D,N], D, dt_bias [D] float32; D, z and
    dt_bias may be None.  ``init``: None or [N,D,N] float32.  ``final``: True (allocate),
    such a tensor to write, or False.  ``chunk_states``: whether to keep what
    selective_scan_bwd needs.  Tokens behind cu_seqlens[N] are not written.
    Returns (y, final, chunk_states)."""
    import torch
    kind, dev = _dtype("x", x), _device("x", x)
    n, T = _sequences(x, cu_seqlens)
    args = _ssm_args(x, dt, A, B, C, D, z, dt_bias)
    width, N = A.shape
    shape, chunks, need, _ = _ssm_plan(kind, n, T, width, N, 1 if softplus else 0, cu_seqlens is not None)
    _maybe("init", init, torch.float32, (n, width, N), dev)
    with _on(dev, stream):
        if out is None:
            out = _like(x)
        else:
            _check("y", out, x.dtype, x.shape, dev)
        final = x.new_empty((n, width, N), dtype=torch.float32) if final is True else None if final is False else final
        _maybe("final", final, torch.float32, (n, width, N), dev)
        states = x.new_empty((chunks, width, N), dtype=torch.float32) if chunk_states else None
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_ssm_fwd(shape, _p(cu_seqlens), *args, _p(init), _p(final), _p(out), _p(states), _p(ws), nbytes,
                                   _current(dev)), "falcon_ssm_fwd")
    return out, final, states


def selective_scan_bwd(x, dt, A, B, C, dy, chunk_states, *, D=None, z=None, dt_bias=None, softplus=True, cu_seqlens=None,
                       init=None, d_final=None, d_init=True, out=None, workspace=None, stream=None):
    """falcon_ssm_bwd on torch tensors: gradients of <dy, y> + <d_final, final> for
    ``selective_scan`` of the same arguments.

    ``chunk_states`` is what ``selective_scan(..., chunk_states=True)`` returned (``init``
    is in it).  dy has the dtype and shape of x; d_final is None or [N,D,N] float32.
    ``d_init``: True (allocate), a [N,D,N] float32 tensor, or False.  ``out``: None or a
    dict of preallocated dx, ddt, dB, dC and, with z, dz (views with dense rows will do).
    Returns dict(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_init): dA [D,N], dD, ddt_bias [D]
    float32, None for what was not given."""
    import torch
    kind, dev = _dtype("x", x), _device("x", x)
    n, T = _sequences(x, cu_seqlens)
    args = _ssm_args(x, dt, A, B, C, D, z, dt_bias)
    width, N = A.shape
    shape, chunks, _, need = _ssm_plan(kind, n, T, width, N, 1 if softplus else 0, cu_seqlens is not None)
    states = (n, width, N)
    _check("dy", dy, x.dtype, x.shape, dev)
    _check("chunk_states", chunk_states, torch.float32, (chunks, width, N), dev)
    for name, t in (("init", init), ("d_final", d_final)):
        _maybe(name, t, torch.float32, states, dev)
    with _on(dev, stream):
        like = dict(dx=x, ddt=dt, dB=B, dC=C, dz=z)
        if out is None:
            out = {k: _like(t) for k, t in like.items() if t is not None}
        rows = {k: _NO_ROWS if t is None else _rows(k, out[k], x.dtype, dev, t.shape) for k, t in like.items()}
        d_init = x.new_empty(states, dtype=torch.float32) if d_init is True else None if d_init is False else d_init
        _maybe("d_init", d_init, torch.float32, states, dev)
        dA = torch.empty_like(A)
        dD, db = (None if t is None else torch.empty_like(t) for t in (D, dt_bias))
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_ssm_bwd(shape, _p(cu_seqlens), *args, _p(chunk_states), _p(dy), _p(d_final), rows["dx"], rows["ddt"],
                                   _p(dA), rows["dB"], rows["dC"], _p(dD), rows["dz"], _p(db), _p(d_init), _p(ws), nbytes,
                                   _current(dev)), "falcon_ssm_bwd")
    return dict(dx=out["dx"], ddt=out["ddt"], dA=dA, dB=out["dB"], dC=out["dC"], dD=dD, dz=None if z is None else out["dz"],
                ddt_bias=db, d_init=d_init)


def selective_scan_step(x, dt, A, B, C, state, *, D=None, z=None, dt_bias=None, softplus=True, state_out=None, out=None,
                        stream=None):
    """falcon_ssm_step: one token of every sequence; x, dt, z [B,D], B, C [B,N], ``state``
    [B,D,N] float32 updated in place, or left as it is with ``state_out``, a tensor for
    the new state.  Returns y [B,D] in the dtype of x."""
    import torch
    kind, dev = _dtype("x", x), _device("x", x)
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [B, D]")
    args = _ssm_args(x, dt, A, B, C, D, z, dt_bias)
    n, (width, N) = x.shape[0], A.shape
    if state_out is None:
        state_out = state
    for name, t in (("state", state), ("state_out", state_out)):
        _check(name, t, torch.float32, (n, width, N), dev)
    with _on(dev, stream):
        if out is None:
            out = _like(x)
        else:
            _check("y", out, x.dtype, x.shape, dev)
        shape, *_ = _ssm_plan(kind, n, 1, width, N, 1 if softplus else 0, False)
        _done(lib().falcon_ssm_step(shape, *args, _p(state), _p(state_out), _p(out), _current(dev)), "falcon_ssm_step")
    return out


# ---- Projections --------------------------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _linear_plan(dtype, tokens, K, N, act, out):
    """(pointer to the C shape, workspace bytes of the forward, of the backward)."""
    shape = LinearShape(dtype, *_ints(tokens, K, N), act, out)
    L, ref = lib(), ctypes.byref(shape)
    return ctypes.pointer(shape), L.falcon_linear_fwd_workspace(ref), L.falcon_linear_bwd_workspace(ref)


@functools.lru_cache(maxsize=None)
def _linear_types(dtype, out_dtype):
    """(C type of the operands, whether 8 bits, type of the result, its C type)."""
    import torch
    f8 = dtype is _f8()
    kind = E4M3 if f8 else _types().get(dtype)
    if kind is None:
        raise TypeError("x must be float32 or bfloat16, or both operands float8_e4m3fn")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if f8 else dtype
    if not f8 and out_dtype is not dtype:
        raise TypeError(f"out_dtype: {out_dtype}, expected {dtype} (only 8-bit operands have another)")
    out = _types().get(out_dtype)
    if out is None:
        raise TypeError("out_dtype must be float32 or bfloat16")
    return kind, f8, out_dtype, out


def _linear_shape(x, weight, activation, out_dtype):
    dev = _device("x", x)
    kind, f8, out_dtype, out = _linear_types(x.dtype, out_dtype)
    size, (*more, K) = weight.shape, x.shape or (None,)
    if len(size) != 2 or size[1] != K:
        raise ValueError(f"x, weight: shapes {tuple(x.shape)}, {tuple(size)}, expected [..., in], [out, in]")
    _check("weight", weight, x.dtype, size, dev)
    plan = _linear_plan(kind, x.numel() // max(K, 1), K, size[0], _activation(activation), out)
    return *plan, tuple(more), out_dtype, f8, dev


def linear(x, weight, *, bias=None, activation=None, residual=None, x_scale=None, weight_scale=None, pre=False,
           out_dtype=None, out=None, workspace=None, stream=None):
    """falcon_linear_fwd on torch tensors: y = act(x weight^T + bias) + residual.

    x [...,in], weight [out,in] (float32 or bfloat16; in a multiple of 16, out of 8; x may be
    a view of a wider projection), bias [out] float32, residual [...,out] like y;
    ``activation``: None, "silu" or "gelu".  Or both float8_e4m3fn, with ``x_scale`` [...] and
    ``weight_scale`` [out] float32 (as ``rms_norm(..., quantize=True)`` and ``quantize_rows``
    give them) and ``out_dtype`` bfloat16 (default) or float32.  ``pre``: whether to return the
    activation's argument [...,out] float32, which linear_bwd needs with an activation (8-bit
    operands are then multiplied as bfloat16, for the fp32 sum).  ``out``: None or a tensor
    for y, which may be the residual.  Returns (y, pre)."""
    import torch
    shape, need, _, lead, odt, f8, dev = _linear_shape(x, weight, activation, out_dtype)
    N = weight.shape[0]
    hx = _rows("x", x, x.dtype, dev)
    full = lead + (N,)
    _maybe("bias", bias, torch.float32, (N,), dev)
    _maybe("residual", residual, odt, full, dev)
    if f8 != (x_scale is not None) or f8 != (weight_scale is not None):
        raise ValueError("x_scale, weight_scale: both for 8-bit operands, and for those only")
    if f8:
        _check("x_scale", x_scale, torch.float32, lead, dev)
        _check("weight_scale", weight_scale, torch.float32, (N,), dev)
    with _on(dev, stream):
        if out is None:
            out = x.new_empty(full, dtype=odt)
        else:
            _check("y", out, odt, full, dev)
        keep = x.new_empty(full, dtype=torch.float32) if pre else None
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_linear_fwd(shape, hx, _p(weight), _p(x_scale), _p(weight_scale), _p(bias), _p(residual), _p(out),
                                      _p(keep), _p(ws), nbytes, _current(dev)), "falcon_linear_fwd")
    return out, keep


def linear_bwd(x, weight, dy, *, pre=None, activation=None, bias=False, dx=True, dweight=True, workspace=None, stream=None):
    """falcon_linear_bwd on torch tensors: gradients of <dy, y> for ``linear`` of the same
    arguments (float32 or bfloat16; the residual's gradient is dy itself).

    dy [...,out] in the dtype of x (a view with dense rows will do); ``pre`` as ``linear(...,
    pre=True)`` returned it, needed with an activation.  ``bias``: whether to return a bias's
    gradient; ``dx``: True (allocate), a tensor to write (a view with dense rows will do) or
    False; ``dweight``: True, a tensor or False.  Returns dict(dx, dweight, dbias): dx and
    dweight in the dtype of x, dbias [out] float32."""
    import torch
    shape, _, need, lead, _, f8, dev = _linear_shape(x, weight, activation, None)
    if f8:
        raise TypeError("x: 8-bit operands have no backward pass")
    N, K = weight.shape
    hx = _rows("x", x, x.dtype, dev)
    hdy = _rows("dy", dy, x.dtype, dev, lead + (N,))
    if activation is not None and pre is None:
        raise ValueError("pre: needed with an activation")
    _maybe("pre", pre, torch.float32, lead + (N,), dev)
    with _on(dev, stream):
        dx = _like(x) if dx is True else None if dx is False else dx
        hdx = _NO_ROWS if dx is None else _rows("dx", dx, x.dtype, dev, x.shape)
        dweight = torch.empty_like(weight) if dweight is True else None if dweight is False else dweight
        _maybe("dweight", dweight, x.dtype, (N, K), dev)
        dbias = torch.empty((N,), dtype=torch.float32, device=dev) if bias else None
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_linear_bwd(shape, hx, _p(weight), _p(pre) if activation is not None else None, hdy, hdx,
                                      _p(dweight), _p(dbias), _p(ws), nbytes, _current(dev)), "falcon_linear_bwd")
    return dict(dx=dx, dweight=dweight, dbias=dbias)
