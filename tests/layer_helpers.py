"""Shared helpers of the layer operators' GPU tests: inputs, and elementwise bounds.

Every bound is derived from what the kernels round, in units of u = 2^-24 (half a step
of fp32) and, for bf16 tensors, of half = eps / 2 = 2^-8 per rounding to bf16.
"""

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126   # the least normal number of fp32 and bf16


def tdt(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def half(dtype):
    """The largest relative error of one rounding to an output's type."""
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def rand(seed, *shape, dtype="fp32", device="cuda", scale=1.0):
    """A normal tensor of the type on the device."""
    import torch
    a = np.random.Generator(np.random.PCG64(seed)).normal(size=shape) * scale
    return torch.from_numpy(a.astype(np.float32)).to(tdt(dtype)).to(device)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def offsets(lens, device="cuda"):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device)


def check(name, got, ref, bound):
    """|got - ref| <= bound everywhere (got, ref, bound broadcast), naming the worst entry."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bound = np.broadcast_to(np.asarray(bound, np.float64), ref.shape)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - ref) - bound
    if over.size and over.max() > 0:
        at = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{name}{list(map(int, at))}: got {got[at]!r}, expected {ref[at]!r}, off by "
                             f"{abs(got[at] - ref[at]):.3e}, bound {bound[at]:.3e}; {np.mean(over > 0):.2%} are over")


# ---- Gated linear recurrence ----------------------------------------------------------
# A step's decay is off by at most (1 + 1 + |g|) 2 u relative (the hardware's exp2 within
# one step, its argument's rounding), forming the input by 3 u, and every product and sum
# by u.  A state is a sum over earlier inputs of products of decays; composing maps instead
# of stepping through them forms the same products, each factor rounded at most 5 times
# over (thread, group, chunk, chunk group, replay).  So an error of C u enters per step,
# relative to the sum H of absolute values, and decays with the state: E_t = lam E + H.
SCAN_C = 16.0


def scan_bounds(x, g, init, mix):
    """(H, E): the scan of absolute values, and the scan of those."""
    from oracle import layer as L
    lam = np.exp(g)
    H, _ = L.gated_scan(np.abs(x) * (1 - lam if mix else 1.0), g, None if init is None else np.abs(init))
    E, _ = L.gated_scan(H, g)
    return H, E * SCAN_C * U


def reverse(a):
    return a[::-1]


def scan_back_bounds(x, g, dh, d_final, init, mix):
    """(bound of r_t, |r|_t) with r_t = lam_t delta_t: the reverse recurrence is the same
    one in reversed time, delta_t = dh_t + lam_{t+1} delta_{t+1}."""
    from oracle import layer as L
    lam = np.exp(g)
    nxt = np.vstack([g[1:], np.zeros((1, g.shape[1]))])     # log decay that delta_{t+1} takes to t
    D, _ = L.gated_scan(reverse(np.abs(dh)), reverse(nxt), None if d_final is None else np.abs(d_final))
    E, _ = L.gated_scan(D, reverse(nxt))
    return reverse(E) * SCAN_C * U, reverse(D), lam


# ---- Attention ---------------------------------------------------------------------------
def attention_bounds(q, k, v, scale, dtype, do=None):
    """Elementwise bounds of o, lse (and dq, dk, dv) of one sequence.

    A score is a sum of d products: off by (d + 2) u times the sum of their absolute
    values, A_ij (one rounding more for the scale); e^s is off by that, by u |s| in its
    argument and by a step of the hardware's exp2.  So a weight is off relatively by
    e_ij = 2 max_j (...) (numerator and normaliser).  bf16 rounds the weights once (half)
    before their products with v.  o is rounded to its type.  In the backward pass D = do.o
    uses the rounded o, P and dS are rounded once before their products, and the gradients
    to their type."""
    from oracle import layer as L
    f = L.attention(q, k, v, scale)
    H, d = q.shape[1:]
    Lk, grp = k.shape[0], H // k.shape[1]
    hb = half(dtype) if dtype == "bf16" else 0.0     # rounding of a weight before a product
    ho = half(dtype)                                 # rounding of a result
    bo, bl = np.zeros_like(f["o"]), np.zeros_like(f["lse"])
    out = dict(f)
    if do is not None:
        gr = L.attention_backward(q, k, v, do, scale)
        out.update(gr)
        bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(H):
        kv = h // grp
        A = scale * (np.abs(q[:, h]) @ np.abs(k[:, kv]).T)
        es = (d + 4) * U * A.max(initial=0.0) + U * (np.abs(A).max(initial=0.0) + 4) * 2
        ep = 2 * es + (Lk + 16) * U                  # relative error of a weight; sums over the keys
        # a weight (and a dS, a result) below the least normal number, TINY, may become 0: an
        # absolute error of TINY.  As ep >= 16 u = 2^-20, ep (p + 2^-100) >= ep p + TINY.
        p = f["p"][h] + 2.0 ** -100
        pv = p @ np.abs(v[:, kv])
        bo[:, h] = (hb + ep) * (1 + ho) * pv + ho * np.abs(f["o"][:, h])
        bl[:, h] = 2 * es + (Lk + 16) * U + 4 * U * np.where(np.isfinite(f["lse"][:, h]), np.abs(f["lse"][:, h]), 0)
        if do is not None:
            g = np.abs(do[:, h])
            bv[:, kv] += (hb + ep) * (p.T @ g)
            dp = g @ np.abs(v[:, kv]).T
            eD = np.sum(g * (bo[:, h] + (d + 2) * U * np.abs(f["o"][:, h])), -1, keepdims=True)
            D = np.sum(g * np.abs(f["o"][:, h]), -1, keepdims=True)
            eds = p * ((d + 4) * U * dp + eD + (ep + 2 * U) * (dp + D)) + hb * np.abs(gr["ds"][h]) + TINY
            bq[:, h] = scale * (eds + (Lk + 2) * U * np.abs(gr["ds"][h])) @ np.abs(k[:, kv])
            bk[:, kv] += scale * (eds + (q.shape[0] * grp + 2) * U * np.abs(gr["ds"][h])).T @ np.abs(q[:, h])
    out.update(bo=bo + TINY, bl=bl)
    if do is not None:
        out.update(bq=bq + ho * np.abs(gr["dq"]) + TINY, bk=bk + ho * np.abs(gr["dk"]) + TINY,
                   bv=bv + ho * np.abs(gr["dv"]) + TINY)
    return out
