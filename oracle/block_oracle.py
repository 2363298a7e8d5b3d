"""fp64 definitions of the operators of a state-space block, one sequence at a time: the norm of
the residual stream, the projections, the short causal convolution and the selective
state-space scan, each with its gradients.  Test infrastructure only."""

import math

import numpy as np

F8_MAX = 448.0


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def activation(p, act):
    """(act(p), act'(p))."""
    if act == "silu":
        s = sigmoid(p)
        return p * s, s * (1 + p * (1 - s))
    if act == "gelu":
        phi = 0.5 * (1 + np.vectorize(math.erf, otypes=[float])(p / math.sqrt(2)))
        return p * phi, phi + p * np.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    return p, np.ones_like(p)


# ---- Norm of the residual stream ------------------------------------------------------

def rms_norm(s, w, eps=1e-6):
    return s * w / np.sqrt((s * s).mean(-1, keepdims=True) + eps)


def rms_norm_backward(s, w, dy, ds=0.0, eps=1e-6):
    """(dx, dw) over rows s [tokens, width]."""
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    v = s * r
    return ds + r * (w * dy - v * (w * dy * v).mean(-1, keepdims=True)), (dy * v).sum(0)


# ---- Short causal convolution -----------------------------------------------------------

def conv(x, w, b, init, act=None):
    """x [T, D], w [D, taps], init [taps - 1, D]: (y, final, pre-activation)."""
    T, W = x.shape[0], w.shape[1]
    ext = np.concatenate([init, x])
    p = b + sum(w[:, j] * ext[j:j + T] for j in range(W))
    return activation(p, act)[0], ext[T:], p


def conv_backward(x, w, b, init, dy, d_final, act=None):
    """dict of dx, dw, db, dinit, d (the gradient of the pre-activation)."""
    T, W = x.shape[0], w.shape[1]
    ext = np.concatenate([init, x])
    d = dy * activation(conv(x, w, b, init)[2], act)[1]
    back = np.zeros_like(ext)
    back[T:] += d_final
    dw = np.zeros_like(w)
    for j in range(W):
        back[j:j + T] += w[:, j] * d
        dw[:, j] = (d * ext[j:j + T]).sum(0)
    return dict(dx=back[W - 1:], dinit=back[:W - 1], dw=dw, db=d.sum(0), d=d)


# ---- Selective state-space scan -----------------------------------------------------------

def steps_of(dt, bias, softplus=True):
    """(delta, its derivative by dt)."""
    raw = dt + bias
    if not softplus:
        return raw, np.ones_like(raw)
    return np.logaddexp(raw, 0), sigmoid(raw)


def ssm(x, dt, A, B, C, D=0.0, z=None, bias=0.0, softplus=True, init=None):
    """x, dt, z [T, D], A, init [D, N], B, C [T, N]: dict of y, final, h [T + 1, D, N], read, delta."""
    T = x.shape[0]
    delta, slope = steps_of(dt, bias, softplus)
    h = np.zeros((T + 1,) + A.shape)
    h[0] = 0 if init is None else init
    read = np.zeros(x.shape)
    for t in range(T):
        h[t + 1] = np.exp(delta[t][:, None] * A) * h[t] + (delta[t] * x[t])[:, None] * B[t]
        read[t] = h[t + 1] @ C[t] + D * x[t]
    y = read if z is None else read * activation(z, "silu")[0]
    return dict(y=y, final=h[T], h=h, read=read, delta=delta, slope=slope)


def ssm_backward(x, dt, A, B, C, dy, D=0.0, z=None, bias=0.0, softplus=True, init=None, d_final=None):
    T = x.shape[0]
    f = ssm(x, dt, A, B, C, D, z, bias, softplus, init)
    delta, h = f["delta"], f["h"]
    gate, gslope = (1.0, None) if z is None else activation(z, "silu")
    gy = dy * gate
    out = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dB=np.zeros_like(B), dC=np.zeros_like(C), dA=np.zeros_like(A),
               dz=None if z is None else dy * f["read"] * gslope, dD=(gy * x).sum(0))
    r = np.zeros_like(A) if d_final is None else d_final.copy()
    for t in range(T - 1, -1, -1):
        g = r + gy[t][:, None] * C[t]
        r = np.exp(delta[t][:, None] * A) * g
        w = r * h[t]
        gb = g @ B[t]
        out["dx"][t] = gb * delta[t] + D * gy[t]
        out["ddt"][t] = ((w * A).sum(-1) + gb * x[t]) * f["slope"][t]
        out["dA"] += w * delta[t][:, None]
        out["dB"][t] = (delta[t] * x[t]) @ g
        out["dC"][t] = gy[t] @ h[t + 1]
    out["dbias"] = out["ddt"].sum(0)
    out["dinit"] = r
    return out


# ---- Projections -----------------------------------------------------------------------------

def linear(x, w, b=0.0, act=None, res=0.0):
    """(y, pre-activation)."""
    p = x @ w.T + b
    return activation(p, act)[0] + res, p


def linear_backward(x, w, dy, p, act=None):
    d = dy * activation(p, act)[1]
    return dict(dx=d @ w, dw=d.T @ x, db=d.sum(0), d=d)
