"""Python binding of the layer operators of libfalcon (include/falcon.h): the gated
linear recurrence, the query / key norm with rotary positions, and causal attention.

Argument marshalling only, as falcon.py: every step of the computation runs in the HIP
kernels.  A call runs on the device of its tensors; ``stream`` (default: that device's
current stream) is a torch stream of the same device, and what the call allocates
belongs to it.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math

from .falcon import OK, AttnShape, FalconError, Heads, QkShape, ScanShape, _check_tensor, lib

SCAN_CHUNK = 256   # FALCON_SCAN_CHUNK
LAYOUTS = {"half": 0, "interleaved": 1}
_HERE = contextlib.nullcontext()

# A small call's time is this module's: checks are written to pass quickly (the long ones in
# falcon.py run only to say what is wrong), and what follows from sizes alone (the C structs,
# the workspace sizes) is kept by sizes.


@functools.lru_cache(maxsize=None)
def _types():
    import torch
    return {torch.float32: 0, torch.bfloat16: 1}


def _dtype(name, t):
    dt = _types().get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return dt


def _device(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name}: must live on a GPU")
    return t.device


def _check(name, t, dtype, shape, dev):
    """_check_tensor, quick where the tensor is as it should be."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check_tensor(name, t, dtype, shape, dev)


def _p(t):
    return None if t is None else t.data_ptr()


def _on(dev, stream):
    """The context of a call: its device current, allocations on the stream it runs on."""
    import torch
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream: must belong to {dev}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


@functools.lru_cache(maxsize=None)
def _raw_stream():
    """device index -> its current HIP stream; by the short way where this torch has one
    (making a stream object takes 2 us)."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)


def _current(dev):
    """The HIP stream of a call, inside its context."""
    return _raw_stream()(dev.index)


def _done(status, where):
    if status != OK:
        raise FalconError(status, where)


def _workspace(need, given, dev):
    """(tensor or None, bytes) of a call that needs ``need`` bytes."""
    import torch
    if given is None:
        return (torch.empty(need, dtype=torch.uint8, device=dev) if need else None), need
    _check_tensor("workspace", given, torch.uint8, (given.numel(),), dev)
    return given, given.numel()


def _offsets(name, cu, dev):
    import torch
    if cu.dim() != 1 or cu.numel() < 2:
        raise ValueError(f"{name}: shape {tuple(cu.shape)}, expected (sequences + 1,)")
    _check(name, cu, torch.int32, cu.shape, dev)
    return cu.numel() - 1


def _ints(*sizes):
    """The sizes, which the C structs hold in 32 bits (ctypes would drop the rest)."""
    if max(sizes) > 2 ** 31 - 1:
        raise ValueError(f"sizes {sizes}: at most 2^31 - 1")
    return sizes


# ---- Gated linear recurrence ----------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _scan_plan(dtype, n, T, D, mix, packed):
    """(pointer to the C shape, workspace bytes)."""
    shape = ScanShape(dtype, *_ints(n, T, D), 1 if mix else 0)
    return ctypes.pointer(shape), lib().falcon_scan_workspace(ctypes.byref(shape), packed)


def _scan_shape(x, log_lambda, cu_seqlens, mix):
    dt, dev = _dtype("x", x), _device("x", x)
    packed = cu_seqlens is not None
    if x.dim() != (2 if packed else 3):
        raise ValueError(f"x: shape {tuple(x.shape)}, expected " + ("[total, D]" if packed else "[B, T, D]"))
    _check("x", x, x.dtype, x.shape, dev)
    _check("log_lambda", log_lambda, x.dtype, x.shape, dev)
    T, D = x.shape[-2:]
    n = _offsets("cu_seqlens", cu_seqlens, dev) if packed else x.shape[0]
    shape, need = _scan_plan(dt, n, T, D, bool(mix), packed)
    return shape, need, n, D, dev


def _states_shape(x, cu_seqlens):
    rows, T = (x.shape[0] if cu_seqlens is None else 1), x.shape[-2]
    return rows, -(-T // SCAN_CHUNK), x.shape[-1]


def gated_scan(x, log_lambda, *, cu_seqlens=None, mix=False, init=None, final=True, chunk_states=False, out=None,
               workspace=None, stream=None):
    """falcon_scan_fwd on torch tensors: h_t = lam_t h_{t-1} + u_t per channel, with
    lam = exp(log_lambda) and u = x, or (1 - lam) x with ``mix``.

    x, log_lambda [B,T,D] (float32 or bfloat16, D a multiple of 8), or [total,D] with
    ``cu_seqlens``, an int32 device tensor [N+1] of token offsets.  ``init``: None or
    [N,D] float32.  ``final``: True (allocate), a [N,D] float32 tensor to write (may be
    ``init``), or False.  ``chunk_states``: whether to keep what gated_scan_bwd needs.
    Tokens behind cu_seqlens[N] are not written.  Returns (h, final, chunk_states)."""
    import torch
    shape, need, n, D, dev = _scan_shape(x, log_lambda, cu_seqlens, mix)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x)
        else:
            _check("h", out, x.dtype, x.shape, dev)
        if final is True:
            final = x.new_empty((n, D), dtype=torch.float32)
        elif final is False:
            final = None
        for name, t in (("init", init), ("final", final)):
            if t is not None:
                _check(name, t, torch.float32, (n, D), dev)
        states = x.new_empty(_states_shape(x, cu_seqlens), dtype=torch.float32) if chunk_states else None
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_scan_fwd(shape, _p(cu_seqlens), _p(x), _p(log_lambda), _p(init), _p(final), _p(out),
                                    _p(states), _p(ws), nbytes, _current(dev)), "falcon_scan_fwd")
    return out, final, states


def gated_scan_bwd(x, log_lambda, dh, chunk_states, *, cu_seqlens=None, mix=False, init=None, d_final=None,
                   d_init=True, out=None, workspace=None, stream=None):
    """falcon_scan_bwd on torch tensors: gradients of <dh, h> + <d_final, final>.

    ``chunk_states`` is what ``gated_scan(..., chunk_states=True)`` returned for the same
    arguments.  dh has the dtype and shape of x; ``d_final`` is None or [N,D] float32.
    ``d_init``: True (allocate), a [N,D] float32 tensor, or False.  ``out``: None or a
    dict of preallocated dx, dg.  Returns dict(dx, dg, d_init)."""
    import torch
    shape, need, n, D, dev = _scan_shape(x, log_lambda, cu_seqlens, mix)
    _check("dh", dh, x.dtype, x.shape, dev)
    _check("chunk_states", chunk_states, torch.float32, _states_shape(x, cu_seqlens), dev)
    with _on(dev, stream):
        if out is None:
            out = dict(dx=torch.empty_like(x), dg=torch.empty_like(x))
        for name in ("dx", "dg"):
            _check(name, out[name], x.dtype, x.shape, dev)
        if d_init is True:
            d_init = x.new_empty((n, D), dtype=torch.float32)
        elif d_init is False:
            d_init = None
        for name, t in (("init", init), ("d_final", d_final), ("d_init", d_init)):
            if t is not None:
                _check(name, t, torch.float32, (n, D), dev)
        ws, nbytes = _workspace(need, workspace, dev)
        _done(lib().falcon_scan_bwd(shape, _p(cu_seqlens), _p(x), _p(log_lambda), _p(init), _p(chunk_states), _p(dh),
                                    _p(d_final), _p(out["dx"]), _p(out["dg"]), _p(d_init), _p(ws), nbytes,
                                    _current(dev)), "falcon_scan_bwd")
    return dict(dx=out["dx"], dg=out["dg"], d_init=d_init)


def gated_scan_step(x, log_lambda, state, *, mix=False, out=None, stream=None):
    """falcon_scan_step: one token; x, log_lambda [B,D], ``state`` [B,D] float32 updated
    in place.  Returns h [B,D] in the dtype of x."""
    import torch
    dt, dev = _dtype("x", x), _device("x", x)
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [B, D]")
    B, D = x.shape
    _check("x", x, x.dtype, (B, D), dev)
    _check("log_lambda", log_lambda, x.dtype, (B, D), dev)
    _check("state", state, torch.float32, (B, D), dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x)
        else:
            _check("h", out, x.dtype, (B, D), dev)
        shape, _ = _scan_plan(dt, B, 1, D, bool(mix), False)
        _done(lib().falcon_scan_step(shape, _p(x), _p(log_lambda), _p(state), _p(out), _current(dev)),
              "falcon_scan_step")
    return out


# ---- Heads ------------------------------------------------------------------------

def _heads(name, t, dtype, dev, shape=None):
    """falcon_heads_t of t [..., heads, d] (of this shape, if given): dense heads, tokens
    one stride apart (views of a wider projection are taken as they are)."""
    size = t.shape
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if len(size) < 3 or (shape is not None and size != shape):
        raise ValueError(f"{name}: shape {tuple(size)}, expected {'[..., heads, d]' if shape is None else tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: must live on {dev}")
    *sizes, H, D = size
    step = H * D                       # the distance of two tokens, if there are two
    if not t.is_contiguous():
        *strides, sh, sd = t.stride()
        want = None
        ok = (sd == 1 or D == 1) and (sh == D or H == 1)
        for n, s in zip(reversed(sizes), reversed(strides)):
            if n == 1:
                continue
            if want is None:
                step = want = s
            ok = ok and s == want
            want = want * n
        if not ok or step < H * D:
            raise ValueError(f"{name}: heads must be dense and tokens one stride apart")
    if (step * t.element_size()) % 16:
        raise ValueError(f"{name}: the distance of two tokens must be a multiple of 16 bytes")
    return Heads(t.data_ptr(), step)


def _dense(t):
    """A new dense tensor like t, and its falcon_heads_t."""
    import torch
    o = torch.empty_like(t, memory_format=torch.contiguous_format)
    return o, Heads(o.data_ptr(), t.shape[-1] * t.shape[-2])


# ---- Query / key norm with rotary positions -----------------------------------------

def rope_frequencies(rot, base=10000.0, *, scaling=None, factor=1.0, original_length=None, beta_fast=32.0,
                     beta_slow=1.0, device=None):
    """(inv_freq, rot_scale) of a rotation of ``rot`` entries: inv_freq [rot / 2] float64
    radians per position, base^(-2 j / rot), scaled for contexts ``factor`` times as long:

    - None: as they are;
    - "linear": positions interpolated, every frequency divided by the factor;
    - "ntk": the base raised to base factor^(rot / (rot - 2)), which leaves the fastest
      pair as it is and divides the slowest by the factor;
    - "parts": the by-parts interpolation of YaRN (Peng et al., 2023): pairs that turn more
      than ``beta_fast`` times in ``original_length`` tokens are kept, those that turn less
      than ``beta_slow`` times are divided by the factor, with a ramp over the pairs between;
      the rotated part is scaled by 0.1 ln(factor) + 1 (a factor of at most 1: by 1)."""
    import torch
    if rot < 2 or rot % 2:
        raise ValueError(f"rot: {rot}, expected a positive even number")
    if not 0 < base < math.inf or not 0 < factor < math.inf:
        raise ValueError("base and factor must be positive and finite")
    j = torch.arange(rot // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("scaling 'ntk' needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-2.0 * j / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        if not original_length or not original_length > 0 or not base > 1 or not beta_fast >= beta_slow > 0:
            raise ValueError("scaling 'parts' needs original_length, a base over 1, and beta_fast >= beta_slow > 0")

        def pair(turns):   # the (fractional) pair that turns so often in original_length tokens
            return rot * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

        # the ramp may end past the last pair (long original contexts, where the slowest pair still
        # turns more than beta_slow times); the method limits its end by rot - 1
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(max(math.ceil(pair(beta_slow)), 0), rot - 1)
        ramp = ((j - low) / max(high - low, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling: {scaling!r}, expected None, 'linear', 'ntk' or 'parts'")
    return freq.to(device) if device is not None else freq, scale


@functools.lru_cache(maxsize=1024)
def _qk_plan(dtype, tokens, hq, hk, d, *rest):
    """(pointer to the C shape, workspace bytes of the backward)."""
    shape = QkShape(dtype, *_ints(tokens, hq, hk, d), *rest)
    return ctypes.pointer(shape), lib().falcon_qk_norm_rope_bwd_workspace(ctypes.byref(shape))


def _qk_shape(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, layout, rot_scale, grad_dtype):
    import torch
    if q.dim() < 3 or k.dim() < 3 or q.shape[:-2] != k.shape[:-2] or q.shape[-1] != k.shape[-1]:
        raise ValueError(f"q, k: shapes {tuple(q.shape)}, {tuple(k.shape)}, expected [..., heads, d] of the same tokens")
    if layout not in LAYOUTS:
        raise ValueError(f"layout: {layout!r}, expected 'half' or 'interleaved'")
    dt, dev = _dtype("q", q), _device("q", q)
    lead, d = q.shape[:-2], q.shape[-1]
    _check("positions", positions, torch.int32, lead, dev)
    tokens = positions.numel()
    rot = 0
    if inv_freq is not None:
        _check("inv_freq", inv_freq, torch.float64, (inv_freq.numel(),), dev)
        rot = 2 * inv_freq.numel()
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if not norm:
                raise ValueError(f"{name}: weights belong to the norm")
            _check(name, w, torch.float32, (d,), dev)
    shape, need = _qk_plan(dt, tokens, q.shape[-2], k.shape[-2], d, rot, LAYOUTS[layout], 1 if norm else 0, float(eps),
                           float(rot_scale), dt if grad_dtype is None else grad_dtype)
    return shape, need, d, dev


def qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, norm=True, eps=1e-6, layout="half",
                 rot_scale=1.0, out=None, stream=None):
    """falcon_qk_norm_rope on torch tensors: every head of q and k divided by its root
    mean square (``norm``; times its weight), then its first 2 * len(inv_freq) entries
    turned by positions * inv_freq.

    q [..., Hq, d], k [..., Hk, d] (float32 or bfloat16; views of a projection's output
    with dense heads will do), positions [...] int32, inv_freq [rot / 2] float64 (None:
    no rotation), weights [d] float32.  ``layout``: "half" (pairs j, j + rot / 2) or
    "interleaved" (2 j, 2 j + 1).  ``out``: None or (q_out, k_out), which may be q and k.
    Returns (q_out, k_out)."""
    shape, _, _, dev = _qk_shape(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, layout, rot_scale, None)
    hq, hk = _heads("q", q, q.dtype, dev), _heads("k", k, q.dtype, dev)
    with _on(dev, stream):
        if out is None:
            (yq, oq), (yk, ok) = _dense(q), _dense(k)
        else:
            yq, yk = out
            oq, ok = _heads("q_out", yq, q.dtype, dev, q.shape), _heads("k_out", yk, q.dtype, dev, k.shape)
        _done(lib().falcon_qk_norm_rope(shape, hq, hk, _p(q_weight), _p(k_weight), _p(positions), _p(inv_freq), oq, ok,
                                        _current(dev)), "falcon_qk_norm_rope")
    return yq, yk


def qk_norm_rope_bwd(q, k, positions, inv_freq, dq_out, dk_out, *, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                     layout="half", rot_scale=1.0, out=None, workspace=None, stream=None):
    """falcon_qk_norm_rope_bwd on torch tensors: gradients of <dq_out, q_out> +
    <dk_out, k_out> for ``qk_norm_rope`` of the same arguments.

    dq_out, dk_out are both in the dtype of q or both float32 (as chunk_bwd gives them).
    ``out``: None or a dict of preallocated dq, dk.  Returns dict(dq, dk, dq_weight,
    dk_weight): dq, dk in the dtype of q, the weights' gradients [d] float32 (None where
    no weight was given)."""
    import torch
    grad = _dtype("dq_out", dq_out)
    shape, need, d, dev = _qk_shape(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, layout, rot_scale, grad)
    hq, hk = _heads("q", q, q.dtype, dev), _heads("k", k, q.dtype, dev)
    gq = _heads("dq_out", dq_out, dq_out.dtype, dev, q.shape)
    gk = _heads("dk_out", dk_out, dq_out.dtype, dev, k.shape)
    with _on(dev, stream):
        if out is None:
            (dq, oq), (dk, ok) = _dense(q), _dense(k)
        else:
            dq, dk = out["dq"], out["dk"]
            oq, ok = _heads("dq", dq, q.dtype, dev, q.shape), _heads("dk", dk, q.dtype, dev, k.shape)
        dwq = q.new_empty((d,), dtype=torch.float32) if q_weight is not None else None
        dwk = q.new_empty((d,), dtype=torch.float32) if k_weight is not None else None
        ws, nbytes = _workspace(need if dwq is not None or dwk is not None else 0, workspace, dev)
        _done(lib().falcon_qk_norm_rope_bwd(shape, hq, hk, _p(q_weight), _p(k_weight), _p(positions), _p(inv_freq), gq,
                                            gk, oq, ok, _p(dwq), _p(dwk), _p(ws), nbytes, _current(dev)),
              "falcon_qk_norm_rope_bwd")
    return dict(dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk)


# ---- Causal attention -----------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _attn_plan(packed, dtype, n, tq, tk, hq, hk, d, scale):
    """(pointer to the C shape, workspace bytes of the forward, of the backward)."""
    shape = AttnShape(dtype, *_ints(n, tq, tk, hq, hk, d), scale)
    L = lib()
    return (ctypes.pointer(shape), L.falcon_attn_fwd_workspace(ctypes.byref(shape), packed),
            L.falcon_attn_bwd_workspace(ctypes.byref(shape), packed))


def _attn_shape(q, k, v, cu_seqlens, cu_seqlens_k, scale):
    dt, dev = _dtype("q", q), _device("q", q)
    dims = 4 if cu_seqlens is None else 3
    if cu_seqlens is None and cu_seqlens_k is not None:
        raise ValueError("cu_seqlens_k: given without cu_seqlens")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != dims:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected " +
                             ("[B, T, heads, d]" if cu_seqlens is None else "[total, heads, d]"))
    (H, d), G = q.shape[-2:], k.shape[-2]
    packed = cu_seqlens is not None
    if not packed:
        n, tq, tk = q.shape[0], q.shape[1], k.shape[1]
    else:
        if cu_seqlens_k is None:
            cu_seqlens_k = cu_seqlens
            if k.shape[0] != q.shape[0]:
                raise ValueError(f"k: {k.shape[0]} tokens, expected {q.shape[0]} (without cu_seqlens_k)")
        n = _offsets("cu_seqlens", cu_seqlens, dev)
        if cu_seqlens_k is not cu_seqlens and _offsets("cu_seqlens_k", cu_seqlens_k, dev) != n:
            raise ValueError("cu_seqlens and cu_seqlens_k differ in length")
        tq, tk = q.shape[0], k.shape[0]
    hq = _heads("q", q, q.dtype, dev)
    hk = _heads("k", k, q.dtype, dev, (tk, G, d) if packed else (n, tk, G, d))
    hv = _heads("v", v, q.dtype, dev, k.shape)
    plan = _attn_plan(packed, dt, n, tq, tk, H, G, d, d ** -0.5 if scale is None else float(scale))
    return plan, cu_seqlens_k, hq, hk, hv, dev


def attention_fwd(q, k, v, *, cu_seqlens=None, cu_seqlens_k=None, scale=None, lse=True, out=None, workspace=None,
                  stream=None):
    """falcon_attn_fwd on torch tensors: causal softmax attention with grouped heads.

    q [B,Tq,Hq,d], k, v [B,Tk,Hk,d] (float32 or bfloat16, Hq a multiple of Hk; views with
    dense heads will do), or packed [total,H,d] with ``cu_seqlens`` (and ``cu_seqlens_k``
    where a sequence's keys are more than its queries, which are then its last tokens),
    int32 device tensors [N+1].  Sequences follow one another without room between them (a
    view of a longer cache is taken for one sequence only).  ``scale``: default d^-1/2.  ``lse``: whether to return
    the log-sum-exp of every row (attention_bwd needs it).
    Returns (o, lse): o like q and dense, lse [..., Hq] float32 or None."""
    import torch
    (shape, fwd_bytes, _), cuk, hq, hk, hv, dev = _attn_shape(q, k, v, cu_seqlens, cu_seqlens_k, scale)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _check("o", out, q.dtype, q.shape, dev)
        rows = q.new_empty(q.shape[:-1], dtype=torch.float32) if lse else None
        ws, nbytes = _workspace(fwd_bytes, workspace, dev)
        _done(lib().falcon_attn_fwd(shape, _p(cu_seqlens), _p(cuk), hq, hk, hv, _p(out), _p(rows),
                                _p(ws), nbytes, _current(dev)), "falcon_attn_fwd")
    return out, rows


def attention_bwd(q, k, v, o, lse, do, *, cu_seqlens=None, cu_seqlens_k=None, scale=None, out=None, workspace=None,
                  stream=None):
    """falcon_attn_bwd on torch tensors: gradients of <do, o> for ``attention_fwd`` of the
    same arguments, which gave o and lse.  ``out``: None or a dict of preallocated dq, dk,
    dv (views with dense heads will do).  Returns dict(dq, dk, dv) in the dtype of q."""
    import torch
    (shape, _, bwd_bytes), cuk, hq, hk, hv, dev = _attn_shape(q, k, v, cu_seqlens, cu_seqlens_k, scale)
    _check("o", o, q.dtype, q.shape, dev)
    _check("lse", lse, torch.float32, q.shape[:-1], dev)
    hdo = _heads("do", do, q.dtype, dev, q.shape)
    with _on(dev, stream):
        if out is None:
            (dq, hdq), (dk, hdk), (dv, hdv) = _dense(q), _dense(k), _dense(v)
        else:
            dq, dk, dv = out["dq"], out["dk"], out["dv"]
            hdq = _heads("dq", dq, q.dtype, dev, q.shape)
            hdk = _heads("dk", dk, q.dtype, dev, k.shape)
            hdv = _heads("dv", dv, q.dtype, dev, k.shape)
        ws, nbytes = _workspace(bwd_bytes, workspace, dev)
        _done(lib().falcon_attn_bwd(shape, _p(cu_seqlens), _p(cuk), hq, hk, hv, _p(o), _p(lse), hdo,
                                hdq, hdk, hdv, _p(ws), nbytes, _current(dev)), "falcon_attn_bwd")
    return dict(dq=dq, dk=dk, dv=dv)
