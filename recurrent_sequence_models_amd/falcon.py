"""Python binding of libfalcon (include/falcon.h): argument marshalling only.

Tensors are torch tensors on the GPU (they supply device memory); the current
torch stream is passed as the HIP stream.  Every step of the computation runs
in the HIP kernels of libfalcon.so; there is no Python or CPU fallback, and a
missing library raises.
"""

from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfalcon.so")

VARIANTS = {"F1": 1, "F1A": 2, "F2": 3, "F2A": 4, "F3": 5, "F3A": 6}
DTYPES = {"fp32": 0, "bf16": 1}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = range(5)
PER_CHANNEL = ("F2", "F2A")
WINDOWED = ("F3", "F3A")

EXPORTS = ("falcon_abi_version", "falcon_status_string", "falcon_chunk_fwd_workspace",
           "falcon_chunk_fwd", "falcon_chunk_fwd_varlen_workspace", "falcon_chunk_fwd_varlen", "falcon_recurrent_step",
           "falcon_chunk_bwd_workspace", "falcon_chunk_bwd",
           "falcon_chunk_fwd_segmented_workspace", "falcon_chunk_fwd_segmented", "falcon_chunk_fwd_static",
           # the layer operators (layer.py)
           "falcon_scan_workspace", "falcon_scan_fwd", "falcon_scan_bwd", "falcon_scan_step",
           "falcon_qk_norm_rope", "falcon_qk_norm_rope_bwd_workspace", "falcon_qk_norm_rope_bwd",
           "falcon_attn_fwd_workspace", "falcon_attn_fwd", "falcon_attn_bwd_workspace", "falcon_attn_bwd",
           # the operators of a state-space block (block.py)
           "falcon_rms_norm", "falcon_rms_norm_bwd_workspace", "falcon_rms_norm_bwd",
           "falcon_conv_fwd", "falcon_conv_bwd_workspace", "falcon_conv_bwd", "falcon_conv_step",
           "falcon_ssm_fwd_workspace", "falcon_ssm_chunks", "falcon_ssm_fwd", "falcon_ssm_bwd_workspace",
           "falcon_ssm_bwd", "falcon_ssm_step",
           "falcon_linear_fwd_workspace", "falcon_linear_fwd", "falcon_linear_bwd_workspace", "falcon_linear_bwd")


class Shape(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("window", ctypes.c_int32), ("eps_gamma", ctypes.c_float),
                ("eps_phi", ctypes.c_float), ("eps_eta", ctypes.c_float), ("align", ctypes.c_int32)]


class State(ctypes.Structure):
    _fields_ = [("S", ctypes.c_void_p), ("x_prev", ctypes.c_void_p),
                ("win_x", ctypes.c_void_p), ("win_v", ctypes.c_void_p)]


class ScanShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("width", ctypes.c_int32), ("input", ctypes.c_int32)]


class QkShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("tokens", ctypes.c_int32), ("heads_q", ctypes.c_int32),
                ("heads_k", ctypes.c_int32), ("d", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rot_scale", ctypes.c_float), ("grad_dtype", ctypes.c_int32)]


class AttnShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("seqlen_q", ctypes.c_int32),
                ("seqlen_k", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32),
                ("d", ctypes.c_int32), ("scale", ctypes.c_float)]


class NormShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("tokens", ctypes.c_int32), ("width", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("out", ctypes.c_int32), ("eps", ctypes.c_float)]


class ConvShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("width", ctypes.c_int32), ("taps", ctypes.c_int32), ("activation", ctypes.c_int32)]


class SsmShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("width", ctypes.c_int32), ("state", ctypes.c_int32), ("softplus", ctypes.c_int32)]


class LinearShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("tokens", ctypes.c_int32), ("in_", ctypes.c_int32), ("out", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class Heads(ctypes.Structure):
    """falcon_heads_t and falcon_heads_out_t: [tokens, heads, d] with a token stride in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64)]


class FalconError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_LIB = None


def lib() -> ctypes.CDLL:
    """Load libfalcon.so (built in-tree by recurrent_sequence_models_amd.build)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() (the HIP "
                               "library is required; there is no fallback)")
        # torch first: its HIP runtime is then the one that libfalcon finds loaded.  The other way
        # round there would be two in the process, and torch's streams are nothing to the second.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        P, I, V, S = ctypes.POINTER, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.falcon_abi_version.restype = I
        L.falcon_abi_version.argtypes = []
        L.falcon_status_string.restype = ctypes.c_char_p
        L.falcon_status_string.argtypes = [I]
        L.falcon_chunk_fwd_workspace.restype = S
        L.falcon_chunk_fwd_workspace.argtypes = [P(Shape)]
        L.falcon_chunk_fwd.restype = I
        L.falcon_chunk_fwd.argtypes = [P(Shape), V, V, V, V, V, P(State), P(State), V, V, V, S, V]
        L.falcon_chunk_fwd_varlen_workspace.restype = S
        L.falcon_chunk_fwd_varlen_workspace.argtypes = [P(Shape)]
        L.falcon_chunk_fwd_varlen.restype = I
        L.falcon_chunk_fwd_varlen.argtypes = [P(Shape), V, V, V, V, V, V, P(State), P(State), V, V, S, V]
        L.falcon_recurrent_step.restype = I
        L.falcon_recurrent_step.argtypes = [P(Shape), V, V, V, V, V, P(State), V, V]
        L.falcon_chunk_fwd_segmented_workspace.restype = S
        L.falcon_chunk_fwd_segmented_workspace.argtypes = [P(Shape), ctypes.c_int32]
        L.falcon_chunk_fwd_segmented.restype = I
        L.falcon_chunk_fwd_segmented.argtypes = [P(Shape), ctypes.c_int32, V, V, V, V, V, P(State), P(State), V, V,
                                                 S, V]
        L.falcon_chunk_fwd_static.restype = I
        L.falcon_chunk_fwd_static.argtypes = [P(Shape), V, V, V, V, V, P(State), P(State), V, V, V]
        L.falcon_chunk_bwd_workspace.restype = S
        L.falcon_chunk_bwd_workspace.argtypes = [P(Shape)]
        L.falcon_chunk_bwd.restype = I
        L.falcon_chunk_bwd.argtypes = [P(Shape), V, V, V, V, V, P(State), V, V, V, V, V, V, V, V, P(State),
                                       V, S, V]
        L.falcon_scan_workspace.restype = S
        L.falcon_scan_workspace.argtypes = [P(ScanShape), I]
        L.falcon_scan_fwd.restype = I
        L.falcon_scan_fwd.argtypes = [P(ScanShape), V, V, V, V, V, V, V, V, S, V]
        L.falcon_scan_bwd.restype = I
        L.falcon_scan_bwd.argtypes = [P(ScanShape), V, V, V, V, V, V, V, V, V, V, V, S, V]
        L.falcon_scan_step.restype = I
        L.falcon_scan_step.argtypes = [P(ScanShape), V, V, V, V, V]
        L.falcon_qk_norm_rope.restype = I
        L.falcon_qk_norm_rope.argtypes = [P(QkShape), Heads, Heads, V, V, V, V, Heads, Heads, V]
        L.falcon_qk_norm_rope_bwd_workspace.restype = S
        L.falcon_qk_norm_rope_bwd_workspace.argtypes = [P(QkShape)]
        L.falcon_qk_norm_rope_bwd.restype = I
        L.falcon_qk_norm_rope_bwd.argtypes = [P(QkShape), Heads, Heads, V, V, V, V, Heads, Heads, Heads, Heads, V, V,
                                              V, S, V]
        L.falcon_attn_fwd_workspace.restype = S
        L.falcon_attn_fwd_workspace.argtypes = [P(AttnShape), I]
        L.falcon_attn_fwd.restype = I
        L.falcon_attn_fwd.argtypes = [P(AttnShape), V, V, Heads, Heads, Heads, V, V, V, S, V]
        L.falcon_attn_bwd_workspace.restype = S
        L.falcon_attn_bwd_workspace.argtypes = [P(AttnShape), I]
        L.falcon_attn_bwd.restype = I
        L.falcon_attn_bwd.argtypes = [P(AttnShape), V, V, Heads, Heads, Heads, V, V, Heads, Heads, Heads, Heads, V, S, V]
        L.falcon_rms_norm.restype = I
        L.falcon_rms_norm.argtypes = [P(NormShape), V, V, V, V, V, V, V]
        L.falcon_rms_norm_bwd_workspace.restype = S
        L.falcon_rms_norm_bwd_workspace.argtypes = [P(NormShape)]
        L.falcon_rms_norm_bwd.restype = I
        L.falcon_rms_norm_bwd.argtypes = [P(NormShape), V, V, V, V, V, V, V, S, V]
        L.falcon_conv_fwd.restype = I
        L.falcon_conv_fwd.argtypes = [P(ConvShape), V, Heads, V, V, V, V, V, V]
        L.falcon_conv_bwd_workspace.restype = S
        L.falcon_conv_bwd_workspace.argtypes = [P(ConvShape), I]
        L.falcon_conv_bwd.restype = I
        L.falcon_conv_bwd.argtypes = [P(ConvShape), V, Heads, V, V, V, V, V, Heads, V, V, V, V, S, V]
        L.falcon_conv_step.restype = I
        L.falcon_conv_step.argtypes = [P(ConvShape), Heads, V, V, V, V, V, V]
        L.falcon_ssm_fwd_workspace.restype = S
        L.falcon_ssm_fwd_workspace.argtypes = [P(SsmShape), I]
        L.falcon_ssm_chunks.restype = I
        L.falcon_ssm_chunks.argtypes = [P(SsmShape), I]
        L.falcon_ssm_fwd.restype = I
        L.falcon_ssm_fwd.argtypes = [P(SsmShape), V, Heads, Heads, V, Heads, Heads, V, Heads, V, V, V, V, V, V, S, V]
        L.falcon_ssm_bwd_workspace.restype = S
        L.falcon_ssm_bwd_workspace.argtypes = [P(SsmShape), I]
        L.falcon_ssm_bwd.restype = I
        L.falcon_ssm_bwd.argtypes = [P(SsmShape), V, Heads, Heads, V, Heads, Heads, V, Heads, V, V, V, V, Heads, Heads, V,
                                     Heads, Heads, V, Heads, V, V, V, S, V]
        L.falcon_ssm_step.restype = I
        L.falcon_ssm_step.argtypes = [P(SsmShape), Heads, Heads, V, Heads, Heads, V, Heads, V, V, V, V, V]
        L.falcon_linear_fwd_workspace.restype = S
        L.falcon_linear_fwd_workspace.argtypes = [P(LinearShape)]
        L.falcon_linear_fwd.restype = I
        L.falcon_linear_fwd.argtypes = [P(LinearShape), Heads, V, V, V, V, V, V, V, V, S, V]
        L.falcon_linear_bwd_workspace.restype = S
        L.falcon_linear_bwd_workspace.argtypes = [P(LinearShape)]
        L.falcon_linear_bwd.restype = I
        L.falcon_linear_bwd.argtypes = [P(LinearShape), Heads, V, V, Heads, Heads, V, V, V, S, V]
        _LIB = L
    return _LIB


def status_string(status: int) -> str:
    return lib().falcon_status_string(int(status)).decode()


ALIGNS = {"prefix": 0, "same": 1}


def make_shape(variant, dtype, batch, seqlen, heads, dk, dv, chunk=64, window=1,
               eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6, align="prefix") -> Shape:
    return Shape(VARIANTS.get(variant, variant) if isinstance(variant, str) else variant,
                 DTYPES.get(dtype, dtype) if isinstance(dtype, str) else dtype,
                 batch, seqlen, heads, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta,
                 ALIGNS.get(align, align) if isinstance(align, str) else align)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _state(st) -> State | None:
    if st is None:
        return None
    return State(st["S"].data_ptr(), st["x_prev"].data_ptr(),
                 st["win_x"].data_ptr() if st.get("win_x") is not None else None,
                 st["win_v"].data_ptr() if st.get("win_v") is not None else None)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_tensor(name, t, dtype, shape, device=None):
    """dtype, shape and contiguity of a tensor, then (unless device is None) that
    it lives on ``device``."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device is not None and (t.device != device or not t.is_cuda):
        raise ValueError(f"{name}: must live on {device}")


def _check_state(name, st, batch, heads, dk, dv, window, device):
    """A state dict the kernels read or write: S [B,H,dv,dk], x_prev [B,H,dk] and,
    for a window of Bw > 1 pairs, win_x [B,H,Bw-1,dk] and win_v [B,H,Bw-1,dv];
    all float32, contiguous, on ``device``.  The library takes raw pointers, so a
    state of another shape would be read or written out of bounds."""
    import torch
    if not isinstance(st, dict):
        raise TypeError(f"{name}: expected a state dict (S, x_prev[, win_x, win_v])")
    need = [("S", (batch, heads, dv, dk)), ("x_prev", (batch, heads, dk))]
    if window > 1:
        need += [("win_x", (batch, heads, window - 1, dk)), ("win_v", (batch, heads, window - 1, dv))]
    for key, _ in need:
        if st.get(key) is None:
            raise ValueError(f"{name}: " + (f"a window of {window} pairs needs '{key}'" if key.startswith("win")
                                            else f"'{key}' is required"))
    for key, shp in need:    # every array's shape first, then where they live
        _check_tensor(f"{name}['{key}']", st[key], torch.float32, shp)
    for key, shp in need:
        _check_tensor(f"{name}['{key}']", st[key], torch.float32, shp, device)


def new_state(batch, heads, dk, dv, window=1, device="cuda"):
    """Zero recurrent state (S, x_prev and, for window > 1, the window pairs)."""
    import torch
    st = dict(S=torch.zeros(batch, heads, dv, dk, device=device),
              x_prev=torch.zeros(batch, heads, dk, device=device))
    if window > 1:
        st["win_x"] = torch.zeros(batch, heads, window - 1, dk, device=device)
        st["win_v"] = torch.zeros(batch, heads, window - 1, dv, device=device)
    return st


def workspace_bytes(variant, dtype, batch, seqlen, heads, dk, dv, chunk=64, window=1, eps_gamma=1e-3,
                    eps_phi=1e-6, eps_eta=1e-6, align="prefix"):
    """falcon_chunk_fwd_workspace for a shape: bytes of scratch that enable the
    two-kernel chunk-parallel path (0: that path is not built for the shape)."""
    shape = make_shape(variant, dtype, batch, seqlen, heads, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta,
                       align)
    return int(lib().falcon_chunk_fwd_workspace(ctypes.byref(shape)))


class ForwardCall:
    """One falcon_chunk_fwd call, validated once and issued as often as needed.

    For loops that run the forward over the same buffers again and again (their
    contents may change between calls): every argument check, allocation and
    ctypes conversion happens here, and each call is one C call.  Arguments are
    those of ``chunk_fwd``; ``stream`` (optional) is fixed for every call unless
    one is passed to ``__call__``.  The object keeps every tensor it passes
    alive: ``out``, ``final`` and ``chunk_states`` are its outputs."""

    def __init__(self, variant, q, k, v, beta, log_lambda, *, chunk=64, window=1, init=None,
                 final=True, chunk_states=False, eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6,
                 out=None, stream=None, workspace=True, align="prefix"):
        import torch
        B, T, H, dk = q.shape
        dv = v.shape[-1]
        dev = q.device
        dt = {torch.float32: "fp32", torch.bfloat16: "bf16"}.get(q.dtype)
        if dt is None:
            raise TypeError("q/k/v must be float32 or bfloat16")
        _check_tensor("q", q, q.dtype, (B, T, H, dk), dev)
        _check_tensor("k", k, q.dtype, (B, T, H, dk), dev)
        _check_tensor("v", v, q.dtype, (B, T, H, dv), dev)
        bshape = (B, T, H, dv) if variant in PER_CHANNEL else (B, T, H)
        _check_tensor("beta", beta, torch.float32, bshape, dev)
        _check_tensor("log_lambda", log_lambda, torch.float32, (B, T, H), dev)
        if out is None:
            out = torch.empty(B, T, H, dv, dtype=q.dtype, device=dev)
        _check_tensor("o", out, q.dtype, (B, T, H, dv), dev)
        if final is True:
            final = new_state(B, H, dk, dv, window if variant in WINDOWED else 1, dev)
        elif final is False:
            final = None
        wst = window if variant in WINDOWED else 1
        if init is not None:
            _check_state("init", init, B, H, dk, dv, wst, dev)
        if final is not None:
            _check_state("final", final, B, H, dk, dv, wst, dev)
        nch = (T + chunk - 1) // chunk
        cs = torch.empty(B, H, nch, dv, dk, dtype=torch.float32, device=dev) if chunk_states else None
        shape = make_shape(variant, dt, B, T, H, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta, align)
        L = lib()
        if workspace is True:
            ws_bytes = L.falcon_chunk_fwd_workspace(ctypes.byref(shape))
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
        elif workspace is False or workspace is None:
            ws, ws_bytes = None, 0
        else:
            _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),), dev)
            ws, ws_bytes = workspace, workspace.numel()
        self.out, self.final, self.chunk_states = out, final, cs
        self._keep = (q, k, v, beta, log_lambda, init, ws)
        self._shape = shape
        self._st_in, self._st_out = _state(init), _state(final)
        self._fn = L.falcon_chunk_fwd
        self._args = (ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(log_lambda),
                      ctypes.byref(self._st_in) if self._st_in else None,
                      ctypes.byref(self._st_out) if self._st_out else None,
                      _ptr(out), _ptr(cs), _ptr(ws), ws_bytes)
        self._stream = None if stream is None else _stream(stream)

    def __call__(self, stream=None):
        st = _stream(stream) if stream is not None else (self._stream if self._stream is not None else _stream(None))
        status = self._fn(*self._args, st)
        if status != OK:
            raise FalconError(status, "falcon_chunk_fwd")
        return self.out, self.final, self.chunk_states


def chunk_fwd(variant, q, k, v, beta, log_lambda, *, chunk=64, window=1, init=None,
              final=True, chunk_states=False, eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6,
              out=None, stream=None, workspace=True, align="prefix"):
    """falcon_chunk_fwd on torch tensors.

    q, k [B,T,H,dk] and v [B,T,H,dv] in float32 or bfloat16; beta [B,T,H] (or
    [B,T,H,dv] for F2/F2A) and log_lambda [B,T,H] float32.  ``init``: None or a
    state dict (S, x_prev, win_x, win_v).  ``final``: True (allocate), a state
    dict to write into (may be ``init``), or False.  ``workspace``: True
    allocates the scratch of the two-kernel chunk-parallel path when the shape
    has one, False runs the one-pass (or fused) kernel without scratch, or a
    uint8 device tensor to use.  ``align``: "prefix" (the pair written at step t
    is (phi(k_{t-1}), v_t)) or "same" ((phi(k_t), v_t)).
    Returns (o, final_state, chunk_states).  For repeated calls over the same
    buffers, ``ForwardCall`` does the checks once."""
    return ForwardCall(variant, q, k, v, beta, log_lambda, chunk=chunk, window=window, init=init, final=final,
                       chunk_states=chunk_states, eps_gamma=eps_gamma, eps_phi=eps_phi, eps_eta=eps_eta, out=out,
                       workspace=workspace, align=align)(stream)


def chunk_fwd_varlen(variant, q, k, v, beta, log_lambda, cu_seqlens, *, chunk=64, window=1, init=None,
                     final=True, eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6, out=None, stream=None,
                     align="prefix", workspace=None):
    """falcon_chunk_fwd_varlen on torch tensors: N packed sequences.

    q, k [total,H,dk] and v [total,H,dv] (float32 or bfloat16); beta [total,H]
    (or [total,H,dv] for F2/F2A) and log_lambda [total,H] float32; cu_seqlens an
    int32 device tensor [N+1] of token offsets.  ``init`` / ``final`` as for
    chunk_fwd, with N sequences.  ``workspace``: None (the one-pass kernel where
    it is built for the shape, else the chunk-parallel path with a workspace
    allocated here), True (allocate and take the chunk-parallel path), False
    (one-pass only), or a uint8 device tensor.  Returns (o, final_state)."""
    import torch
    total, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    N = cu_seqlens.numel() - 1
    dt = {torch.float32: "fp32", torch.bfloat16: "bf16"}.get(q.dtype)
    if dt is None:
        raise TypeError("q/k/v must be float32 or bfloat16")
    _check_tensor("q", q, q.dtype, (total, H, dk), dev)
    _check_tensor("k", k, q.dtype, (total, H, dk), dev)
    _check_tensor("v", v, q.dtype, (total, H, dv), dev)
    _check_tensor("beta", beta, torch.float32, (total, H, dv) if variant in PER_CHANNEL else (total, H), dev)
    _check_tensor("log_lambda", log_lambda, torch.float32, (total, H), dev)
    _check_tensor("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    if out is None:
        out = torch.empty(total, H, dv, dtype=q.dtype, device=dev)
    _check_tensor("o", out, q.dtype, (total, H, dv), dev)
    if final is True:
        final = new_state(N, H, dk, dv, window if variant in WINDOWED else 1, dev)
    elif final is False:
        final = None
    wst = window if variant in WINDOWED else 1
    if init is not None:
        _check_state("init", init, N, H, dk, dv, wst, dev)
    if final is not None:
        _check_state("final", final, N, H, dk, dv, wst, dev)
    shape = make_shape(variant, dt, N, total, H, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta, align)
    L = lib()
    need = int(L.falcon_chunk_fwd_varlen_workspace(ctypes.byref(shape)))
    st_in, st_out = _state(init), _state(final)

    def run(ws):
        return L.falcon_chunk_fwd_varlen(ctypes.byref(shape), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(beta), _ptr(log_lambda),
                                         ctypes.byref(st_in) if st_in else None,
                                         ctypes.byref(st_out) if st_out else None,
                                         _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))

    if workspace is None:
        # the one-pass kernel where it is built; a shape it does not build is refused
        # on the host with FALCON_ERR_WORKSPACE, and then runs with a workspace
        status = run(None)
        if status == ERR_WORKSPACE and need:
            status = run(torch.empty(need, dtype=torch.uint8, device=dev))
    elif workspace is True:
        status = run(torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    elif workspace is False:
        status = run(None)
    else:
        _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),), dev)
        status = run(workspace)
    if status != OK:
        raise FalconError(status, "falcon_chunk_fwd_varlen")
    return out, final


def recurrent_step(variant, q, k, v, beta, log_lambda, state, *, window=1, eps_gamma=1e-3,
                   eps_phi=1e-6, eps_eta=1e-6, out=None, stream=None, align="prefix"):
    """falcon_recurrent_step: one token for every (b, h); ``state`` is updated in place.

    q, k [B,H,dk], v [B,H,dv] (float32 or bfloat16); beta [B,H] (or [B,H,dv]),
    log_lambda [B,H] float32.  Returns o [B,H,dv]."""
    import torch
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    dt = {torch.float32: "fp32", torch.bfloat16: "bf16"}.get(q.dtype)
    if dt is None:
        raise TypeError("q/k/v must be float32 or bfloat16")
    _check_tensor("q", q, q.dtype, (B, H, dk), dev)
    _check_tensor("k", k, q.dtype, (B, H, dk), dev)
    _check_tensor("v", v, q.dtype, (B, H, dv), dev)
    _check_tensor("beta", beta, torch.float32, (B, H, dv) if variant in PER_CHANNEL else (B, H), dev)
    _check_tensor("log_lambda", log_lambda, torch.float32, (B, H), dev)
    _check_state("state", state, B, H, dk, dv, window if variant in WINDOWED else 1, dev)
    if out is None:
        out = torch.empty(B, H, dv, dtype=q.dtype, device=dev)
    _check_tensor("o", out, q.dtype, (B, H, dv), dev)
    shape = make_shape(variant, dt, B, 1, H, dk, dv, 64, window, eps_gamma, eps_phi, eps_eta, align)
    st = _state(state)
    status = lib().falcon_recurrent_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                         _ptr(log_lambda), ctypes.byref(st), _ptr(out), _stream(stream))
    if status != OK:
        raise FalconError(status, "falcon_recurrent_step")
    return out


def bwd_workspace_bytes(variant, dtype, batch, seqlen, heads, dk, dv, chunk=64, eps_gamma=1e-3, eps_phi=1e-6,
                        eps_eta=1e-6, align="prefix", window=1):
    """falcon_chunk_bwd_workspace for a shape (0: the backward pass is not built for it)."""
    shape = make_shape(variant, dtype, batch, seqlen, heads, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta,
                       align)
    return int(lib().falcon_chunk_bwd_workspace(ctypes.byref(shape)))


def chunk_bwd(variant, q, k, v, beta, log_lambda, do, chunk_states, *, init=None, dS_T=None, chunk=64,
              window=1, eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6, align="prefix", d_init=True, out=None,
              workspace=None, stream=None):
    """falcon_chunk_bwd on torch tensors: gradients of <do, o> + <dS_T, S_T>.

    ``chunk_states`` is what ``chunk_fwd(..., chunk_states=True)`` returned for
    the same inputs, ``init`` and ``window``.  ``do`` has the dtype of q; ``dS_T``
    is None or [B,H,dv,dk] float32.  ``d_init``: True (allocate), a state dict to
    write, or False.  ``out``: None or a dict of preallocated dq, dk, dv, dbeta,
    dg.  ``workspace``: None (allocate) or a uint8 device tensor.
    Returns dict(dq, dk, dv, dbeta, dg, dS0, dx_prev0) and, for a window of
    B_w > 1 pairs, dwin_x0 and dwin_v0 (the state entries None when ``d_init``
    is False)."""
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    dt = {torch.float32: "fp32", torch.bfloat16: "bf16"}.get(q.dtype)
    if dt is None:
        raise TypeError("q/k/v must be float32 or bfloat16")
    _check_tensor("q", q, q.dtype, (B, T, H, dk), dev)
    _check_tensor("k", k, q.dtype, (B, T, H, dk), dev)
    _check_tensor("v", v, q.dtype, (B, T, H, dv), dev)
    _check_tensor("do", do, q.dtype, (B, T, H, dv), dev)
    bshape = (B, T, H, dv) if variant in PER_CHANNEL else (B, T, H)
    _check_tensor("beta", beta, torch.float32, bshape, dev)
    _check_tensor("log_lambda", log_lambda, torch.float32, (B, T, H), dev)
    nch = (T + chunk - 1) // chunk
    _check_tensor("chunk_states", chunk_states, torch.float32, (B, H, nch, dv, dk), dev)
    if dS_T is not None:
        _check_tensor("dS_T", dS_T, torch.float32, (B, H, dv, dk), dev)
    if out is None:
        out = dict(dq=torch.empty(B, T, H, dk, device=dev), dk=torch.empty(B, T, H, dk, device=dev),
                   dv=torch.empty(B, T, H, dv, device=dev), dbeta=torch.empty(*bshape, device=dev),
                   dg=torch.empty(B, T, H, device=dev))
    for name, shp in (("dq", (B, T, H, dk)), ("dk", (B, T, H, dk)), ("dv", (B, T, H, dv)),
                      ("dbeta", bshape), ("dg", (B, T, H))):
        _check_tensor(name, out[name], torch.float32, shp, dev)
    wst = window if variant in WINDOWED else 1
    if d_init is True:
        d_init = new_state(B, H, dk, dv, wst, dev)
    elif d_init is False:
        d_init = None
    if init is not None:
        _check_state("init", init, B, H, dk, dv, wst, dev)
    if d_init is not None:
        _check_state("d_init", d_init, B, H, dk, dv, wst, dev)
    shape = make_shape(variant, dt, B, T, H, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta, align)
    L = lib()
    need = int(L.falcon_chunk_bwd_workspace(ctypes.byref(shape)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),), dev)
    st_in, st_d = _state(init), _state(d_init)
    status = L.falcon_chunk_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(log_lambda),
                                ctypes.byref(st_in) if st_in else None, _ptr(chunk_states), _ptr(do), _ptr(dS_T),
                                _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dbeta"]),
                                _ptr(out["dg"]), ctypes.byref(st_d) if st_d else None,
                                _ptr(workspace), workspace.numel(), _stream(stream))
    if status != OK:
        raise FalconError(status, "falcon_chunk_bwd")
    res = dict(out)
    res["dS0"] = d_init["S"] if d_init else None
    res["dx_prev0"] = d_init["x_prev"] if d_init else None
    if wst > 1:
        res["dwin_x0"] = d_init["win_x"] if d_init else None
        res["dwin_v0"] = d_init["win_v"] if d_init else None
    return res


def segmented_workspace_bytes(variant, dtype, batch, seqlen, heads, dk, dv, nseg, chunk=64, window=1,
                              eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6, align="prefix"):
    """falcon_chunk_fwd_segmented_workspace (0: not built for the shape or nseg)."""
    shape = make_shape(variant, dtype, batch, seqlen, heads, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta,
                       align)
    return int(lib().falcon_chunk_fwd_segmented_workspace(ctypes.byref(shape), int(nseg)))


def chunk_fwd_segmented(variant, q, k, v, beta, log_lambda, nseg, *, chunk=64, window=1, init=None, final=True,
                        eps_gamma=1e-3, eps_phi=1e-6, eps_eta=1e-6, out=None, workspace=None, stream=None,
                        align="prefix"):
    """falcon_chunk_fwd_segmented on torch tensors: the chunked forward with every
    sequence cut into ``nseg`` segments run in parallel (T % nseg == 0).  Same
    arguments as ``chunk_fwd``; ``workspace`` is None (allocate) or a uint8 device
    tensor.  Returns (o, final_state)."""
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    dt = {torch.float32: "fp32", torch.bfloat16: "bf16"}.get(q.dtype)
    if dt is None:
        raise TypeError("q/k/v must be float32 or bfloat16")
    _check_tensor("q", q, q.dtype, (B, T, H, dk), dev)
    _check_tensor("k", k, q.dtype, (B, T, H, dk), dev)
    _check_tensor("v", v, q.dtype, (B, T, H, dv), dev)
    bshape = (B, T, H, dv) if variant in PER_CHANNEL else (B, T, H)
    _check_tensor("beta", beta, torch.float32, bshape, dev)
    _check_tensor("log_lambda", log_lambda, torch.float32, (B, T, H), dev)
    if out is None:
        out = torch.empty(B, T, H, dv, dtype=q.dtype, device=dev)
    _check_tensor("o", out, q.dtype, (B, T, H, dv), dev)
    if final is True:
        final = new_state(B, H, dk, dv, window if variant in WINDOWED else 1, dev)
    elif final is False:
        final = None
    wst = window if variant in WINDOWED else 1
    if init is not None:
        _check_state("init", init, B, H, dk, dv, wst, dev)
    if final is not None:
        _check_state("final", final, B, H, dk, dv, wst, dev)
    shape = make_shape(variant, dt, B, T, H, dk, dv, chunk, window, eps_gamma, eps_phi, eps_eta, align)
    L = lib()
    need = int(L.falcon_chunk_fwd_segmented_workspace(ctypes.byref(shape), int(nseg)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),), dev)
    st_in, st_out = _state(init), _state(final)
    status = L.falcon_chunk_fwd_segmented(ctypes.byref(shape), int(nseg), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                          _ptr(log_lambda), ctypes.byref(st_in) if st_in else None,
                                          ctypes.byref(st_out) if st_out else None, _ptr(out), _ptr(workspace),
                                          workspace.numel(), _stream(stream))
    if status != OK:
        raise FalconError(status, "falcon_chunk_fwd_segmented")
    return out, final
