"""Plain fp64 oracles of the layer operators (TEST INFRASTRUCTURE ONLY): the gated linear
recurrence, the query / key norm with rotary positions, and causal attention, each with
its gradients.  They follow the definitions step by step and share no code with the HIP
path; ``tests/test_layer_oracle_pins.py`` ties them to closed forms and differences.

Sequences are given as lists of (begin, end) token ranges, so packed batches are plain
slices of the token axis.
"""

from __future__ import annotations

import numpy as np


def ranges(lens):
    """Token ranges of packed sequences of these lengths."""
    cu = np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))])
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


# ---- Gated linear recurrence ------------------------------------------------------

def gated_scan(x, g, init=None, mix=False):
    """One sequence x, g [T, D]: (h [T, D], final [D])."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    s = np.zeros(x.shape[1]) if init is None else np.array(init, np.float64)
    h = np.empty_like(x)
    for t in range(x.shape[0]):
        lam = np.exp(g[t])
        s = lam * s + (-np.expm1(g[t]) * x[t] if mix else x[t])
        h[t] = s
    return h, s


def gated_scan_backward(x, g, dh, d_final=None, init=None, mix=False):
    """Gradients of <dh, h> + <d_final, final>: dict(dx, dg, d_init)."""
    x, g, dh = (np.asarray(a, np.float64) for a in (x, g, dh))
    T, D = x.shape
    h, _ = gated_scan(x, g, init, mix)
    s0 = np.zeros(D) if init is None else np.asarray(init, np.float64)
    r = np.zeros(D) if d_final is None else np.array(d_final, np.float64)
    dx, dg = np.empty_like(x), np.empty_like(x)
    for t in range(T - 1, -1, -1):
        prev = h[t - 1] if t else s0
        delta, lam = dh[t] + r, np.exp(g[t])
        dx[t] = delta * (-np.expm1(g[t])) if mix else delta
        dg[t] = lam * delta * (prev - x[t] if mix else prev)
        r = lam * delta
    return dict(dx=dx, dg=dg, d_init=r)


# ---- Query / key norm with rotary positions -----------------------------------------

def _pairs(rot, layout):
    j = np.arange(rot // 2)
    return (j, j + rot // 2) if layout == "half" else (2 * j, 2 * j + 1)


def rotate(z, pos, freq, layout="half", scale=1.0):
    """z [N, H, d] with its first 2 len(freq) entries turned by pos [N] * freq."""
    z = np.array(z, np.float64)
    a, b = _pairs(2 * len(freq), layout)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = np.cos(ang) * scale, np.sin(ang) * scale
    za, zb = z[..., a].copy(), z[..., b].copy()
    z[..., a], z[..., b] = za * c - zb * s, zb * c + za * s
    return z


def norm_rope(x, w, pos, freq, norm=True, eps=1e-6, layout="half", scale=1.0):
    x = np.asarray(x, np.float64)
    if norm:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * (1.0 if w is None else np.asarray(w, np.float64))
    return rotate(x, pos, freq, layout, scale)


def norm_rope_backward(x, w, pos, freq, dy, norm=True, eps=1e-6, layout="half", scale=1.0):
    """(dx, dw) of <dy, norm_rope(x)>."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    a, b = _pairs(2 * len(freq), layout)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = np.cos(ang) * scale, np.sin(ang) * scale
    u = dy.copy()
    u[..., a], u[..., b] = dy[..., a] * c + dy[..., b] * s, dy[..., b] * c - dy[..., a] * s
    if not norm:
        return u, None
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    dw = np.sum(u * x * r, (0, 1))
    dx = r * (w * u) - x * r ** 3 * np.mean(w * u * x, -1, keepdims=True)
    return dx, dw


# ---- Causal attention ------------------------------------------------------------------

def attention(q, k, v, scale=None):
    """One sequence: q [Lq, Hq, d], k, v [Lk, Hk, d], the queries the last Lq tokens.
    Returns dict(o, lse, p) with p [Hq, Lq, Lk] the weights."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    Lq, H, d = q.shape
    Lk, grp = k.shape[0], H // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, lse, p = np.zeros_like(q), np.full((Lq, H), -np.inf), np.zeros((H, Lq, Lk))
    for h in range(H):
        for i in range(Lq):
            see = i + Lk - Lq + 1          # keys 0 .. see - 1
            if see <= 0:
                continue
            s = scale * (k[:see, h // grp] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            p[h, i, :see] = e / e.sum()
            lse[i, h] = m + np.log(e.sum())
            o[i, h] = p[h, i, :see] @ v[:see, h // grp]
    return dict(o=o, lse=lse, p=p)


def attention_backward(q, k, v, do, scale=None):
    """Gradients of <do, o>: dict(dq, dk, dv, ds) with ds [Hq, Lq, Lk] those of the
    scaled scores."""
    q, k, v, do = (np.asarray(a, np.float64) for a in (q, k, v, do))
    H, d = q.shape[1:]
    grp = H // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    f = attention(q, k, v, scale)
    dq, dk, dv, ds = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(f["p"])
    for h in range(H):
        p, kv = f["p"][h], h // grp
        dv[:, kv] += p.T @ do[:, h]
        dp = do[:, h] @ v[:, kv].T
        ds[h] = p * (dp - np.sum(do[:, h] * f["o"][:, h], -1, keepdims=True))
        dq[:, h] = scale * ds[h] @ k[:, kv]
        dk[:, kv] += scale * ds[h].T @ q[:, h]
    return dict(dq=dq, dk=dk, dv=dv, ds=ds)
