"""GPU tests of the selective state-space scan, forward, backward and for single tokens,
elementwise against the fp64 definition.

Bounds, with u = 2^-24.  raw = dt + bias is off by u |raw|, softplus by 12 u more: delta is off by
e = (|raw| + 16) u relative (softplus' <= softplus near and below 0, and <= 1 above).  A decay is off by
|delta A| (e + 3 u) + 2 u relative, and composing the steps of a wave, a tile and a segment forms each product at
most a few times over: an error of 8 times that enters a state a step, relative to the scan H of
absolute values, and decays with it.  The reverse scan is bounded the same way, sums add u a term, results
are rounded once (half)."""

import numpy as np
import pytest

from block_helpers import TINY, U, check, f64, half, offsets, rand, same_in_graph, split, strided
from oracle import block as O

pytestmark = pytest.mark.gpu

NAMES = ("x", "dt", "B", "C", "z", "dy")


def inputs(seed, lead, n, D, N, dtype, gate=True, state=True, extras=True):
    """The tensors of a call: dict."""
    import torch
    r = dict(x=rand(seed, *lead, D, dtype=dtype), dt=rand(seed + 1, *lead, D, dtype=dtype, scale=0.7),
             B=rand(seed + 2, *lead, N, dtype=dtype), C=rand(seed + 3, *lead, N, dtype=dtype),
             z=rand(seed + 4, *lead, D, dtype=dtype) if gate else None, dy=rand(seed + 5, *lead, D, dtype=dtype))
    r["A"] = -torch.exp(0.5 * rand(seed + 6, D, N)) * torch.linspace(0.2, 4, N, device="cuda")
    r["D"] = rand(seed + 7, D) if extras else None
    r["bias"] = rand(seed + 8, D) - 2 if extras else None
    r["init"] = rand(seed + 9, n, D, N) if state else None
    r["d_final"] = rand(seed + 10, n, D, N) if state else None
    return r


def reference(a, lens, dtype, softplus, back=True):
    """Values and bounds, one sequence after the other: lists of dicts."""
    D, N = a["A"].shape
    flat = {k: None if a[k] is None else split(f64(a[k]).reshape(-1, a[k].shape[-1]), lens) for k in NAMES}
    A = f64(a["A"])
    skip, bias = (np.zeros(D) if a[k] is None else f64(a[k]) for k in ("D", "bias"))
    out = []
    for i, T in enumerate(lens):
        x, dt, B, C, dy = (flat[k][i] for k in ("x", "dt", "B", "C", "dy"))
        z = None if flat["z"] is None else flat["z"][i]
        h0, rf = (np.zeros((D, N)) if a[k] is None else f64(a[k])[i] for k in ("init", "d_final"))
        f = O.ssm(x, dt, A, B, C, skip, z, bias, softplus, h0)
        raw, delta = dt + bias, f["delta"]
        ed = ((np.abs(raw) + 16) if softplus else 2 + np.abs(raw) / np.maximum(np.abs(delta), 1e-30)) * U
        dl = np.abs(delta)
        dec = np.exp(delta[..., None] * A)
        arel = 8 * ((dl[..., None] * np.abs(A)) * (ed[..., None] + 3 * U) + 4 * U + ed[..., None])
        H, E = np.zeros_like(f["h"]), np.zeros_like(f["h"])
        H[0] = np.abs(h0)
        for t in range(T):
            H[t + 1] = dec[t] * H[t] + (dl[t] * np.abs(x[t]))[:, None] * np.abs(B[t])
            E[t + 1] = dec[t] * E[t] + arel[t] * H[t + 1] + TINY
        read = np.einsum("tdn,tn->td", H[1:], np.abs(C)) + np.abs(skip * x)
        er = np.einsum("tdn,tn->td", E[1:], np.abs(C)) + (N + 6) * U * read
        gate, gs = (1.0, None) if z is None else O.activation(z, "silu")
        eg = 0.0 if z is None else (2 * np.abs(z) + 14) * U
        r = dict(y=f["y"], by=np.abs(gate) * (er + eg * read) + half(dtype) * np.abs(f["y"]) + TINY, final=f["final"], bfinal=E[T])
        if back:
            g = O.ssm_backward(x, dt, A, B, C, dy, skip, z, bias, softplus, h0, rf)
            r.update(g)
            gy = np.abs(dy * gate)
            egy = gy * eg
            G, EG = np.abs(rf), np.zeros((D, N))
            for k in ("dx", "ddt", "dz", "dB", "dC"):
                r["b" + k] = None if g[k] is None else np.zeros_like(g[k])
            r["bdA"], r["bdD"], r["bdbias"] = np.zeros((D, N)), ((T + 64) * U * gy * np.abs(x) + egy * np.abs(x)).sum(0), np.zeros(D)
            many = (min(T, 200) + 120) * U
            for t in range(T - 1, -1, -1):
                Gt = G + gy[t][:, None] * np.abs(C[t])
                Et = EG + egy[t][:, None] * np.abs(C[t]) + 2 * U * Gt
                G, EG = dec[t] * Gt, dec[t] * Et + arel[t] * dec[t] * Gt + TINY
                w, ew = G * H[t], EG * H[t] + G * E[t] + 2 * U * G * H[t] + TINY
                gb, egb = Gt @ np.abs(B[t]), Et @ np.abs(B[t]) + (N + 2) * U * (Gt @ np.abs(B[t]))
                r["bdx"][t] = dl[t] * egb + gb * dl[t] * (ed[t] + 2 * U) + np.abs(skip) * (egy[t] + 2 * U * gy[t])
                S = (w * np.abs(A)).sum(-1) + gb * np.abs(x[t])
                e = (ew * np.abs(A)).sum(-1) + (N + 4) * U * (w * np.abs(A)).sum(-1) + egb * np.abs(x[t]) + 2 * U * S
                eddt = f["slope"][t] * (e + S * (2 * np.abs(raw[t]) + 14) * U)
                r["bddt"][t] = eddt
                r["bdbias"] += eddt + many * np.abs(f["slope"][t]) * S
                r["bdA"] += ew * dl[t][:, None] + w * dl[t][:, None] * (ed[t][:, None] + 4 * U + many)
                ux = dl[t] * np.abs(x[t])
                r["bdB"][t] = ux @ Et + (ux * (ed[t] + 3 * U + (D / 32 + 40) * U)) @ Gt
                r["bdC"][t] = gy[t] @ E[t + 1] + (egy[t] + (D / 32 + 42) * U * gy[t]) @ H[t + 1]
            if z is not None:
                r["bdz"] = np.abs(dy * gs) * er + np.abs(dy) * read * (4 * np.abs(z) + 20) * U
            for k in ("dx", "ddt", "dz", "dB", "dC"):
                if g[k] is not None:
                    r["b" + k] += half(dtype) * np.abs(g[k]) + TINY
            r["bdinit"] = EG
        out.append(r)
    return out


def run(a, cu, softplus, view=False, **kw):
    import torch
    import recurrent_sequence_models_amd as rsm
    v = {k: strided(t) if view and t is not None else t for k, t in a.items() if k in NAMES and k != "dy"}
    args = v["x"], v["dt"], a["A"], v["B"], v["C"]
    opt = dict(D=a["D"], z=v["z"], dt_bias=a["bias"], softplus=softplus, cu_seqlens=cu, init=a["init"], **kw)
    y, final, states = rsm.selective_scan(*args, chunk_states=True, **opt)
    out = None
    if view:
        out = {"d" + k: strided(torch.empty_like(a[k])) for k in ("x", "dt", "B", "C", "z") if a[k] is not None}
    g = rsm.selective_scan_bwd(*args, a["dy"], states, d_final=a["d_final"], out=out, **opt)
    return y, final, g


def compare(a, lens, dtype, softplus, got):
    y, final, g = got
    D = a["A"].shape[0]
    ref = reference(a, lens, dtype, softplus)
    cat = lambda k: np.concatenate([r[k] for r in ref])              # noqa: E731
    stack = lambda k: np.stack([r[k] for r in ref])                  # noqa: E731
    total = sum(lens)
    flat = lambda t: f64(t).reshape(-1, t.shape[-1])[:total]         # noqa: E731
    check("y", flat(y), cat("y"), cat("by"))
    check("final", f64(final), stack("final"), stack("bfinal"))
    for k in ("dx", "ddt", "dB", "dC") + (("dz",) if a["z"] is not None else ()):
        check(k, flat(g[k]), cat(k), cat("b" + k))
    n = len(lens)
    for k, name in (("dA", "dA"), ("dD", "dD"), ("dbias", "ddt_bias")):
        if g[name] is not None:
            check(name, f64(g[name]), sum(r[k] for r in ref),
                  sum(r["b" + k] for r in ref) + (n + 4) * U * sum(np.abs(r[k]) for r in ref) + TINY)
    check("d_init", f64(g["d_init"]), stack("dinit"), stack("bdinit") + TINY)
    assert (g["dz"] is None) == (a["z"] is None) and g["dA"].shape == (D, a["A"].shape[1])


LENS = [[1], [17], [3, 1, 64, 65], [0, 5, 0, 0, 130, 1, 0], [300, 2, 129], [600], [1] * 30, [64, 16, 128, 48]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:7])))
@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("fp32", 16), ("fp32", 32), ("bf16", 64)])
def test_packed(dtype, N, lens):
    a = inputs(1, (sum(lens),), len(lens), 40, N, dtype)
    compare(a, lens, dtype, True, run(a, offsets(lens), True))


@pytest.mark.parametrize("B,T,D,N", [(1, 1, 8, 16), (3, 2, 64, 32), (2, 65, 72, 16), (2, 20, 1000, 64), (5, 257, 32, 16),
                                     (1, 1000, 8, 32)])
@pytest.mark.parametrize("dtype,gate,state,softplus,view", [("bf16", True, False, True, True), ("fp32", False, True, True, False),
                                                            ("fp32", True, True, False, True)])
def test_batch(dtype, B, T, D, N, gate, state, softplus, view):
    a = inputs(20, (B, T), B, D, N, dtype, gate, state, extras=softplus)
    if not softplus:
        a["dt"] = a["dt"].abs() * 0.3
    compare(a, [T] * B, dtype, softplus, run(a, None, softplus, view))


def test_gradients_are_those_of_differences():
    r = np.random.default_rng(3)
    T, D, N = 5, 3, 4
    v = dict(x=r.normal(size=(T, D)), dt=r.normal(size=(T, D)), A=-np.exp(r.normal(size=(D, N))), B=r.normal(size=(T, N)),
             C=r.normal(size=(T, N)), D=r.normal(size=D), z=r.normal(size=(T, D)), bias=r.normal(size=D),
             init=r.normal(size=(D, N)))
    dy, df = r.normal(size=(T, D)), r.normal(size=(D, N))
    g = O.ssm_backward(dy=dy, d_final=df, **v)

    def f(**w):
        o = O.ssm(**w)
        return (dy * o["y"]).sum() + (df * o["final"]).sum()
    for k in v:
        d, h = r.normal(size=v[k].shape), 1e-6
        num = (f(**{**v, k: v[k] + h * d}) - f(**{**v, k: v[k] - h * d})) / (2 * h)
        assert abs(num - (g["d" + k] * d).sum()) < 1e-6, k


@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("fp32", 32), ("fp32", 64)])
def test_single_tokens_continue_a_prompt(dtype, N):
    """Against the whole sequence's outputs and states, within both sides' bounds; in place or not, the same bits."""
    import torch
    import recurrent_sequence_models_amd as rsm
    B, T, D, cut = 3, 40, 72, 33
    a = inputs(40, (B, T), B, D, N, dtype)
    ref = reference(a, [T] * B, dtype, True, back=False)
    args = lambda t: [strided(a[k][:, t].contiguous()) for k in ("x", "dt")] + [a["A"]] + [strided(a[k][:, t].contiguous()) for k in ("B", "C")]  # noqa: E731
    opt = dict(D=a["D"], dt_bias=a["bias"])
    head = {k: a[k][:, :cut].contiguous() for k in ("x", "dt", "B", "C", "z")}
    _, state, none = rsm.selective_scan(head["x"], head["dt"], a["A"], head["B"], head["C"], z=head["z"], init=a["init"], **opt)
    assert none is None
    for t in range(cut, T):
        zt = strided(a["z"][:, t].contiguous())
        kept, other = state.clone(), torch.empty_like(state)
        y = rsm.selective_scan_step(*args(t), state, z=zt, state_out=other, **opt)
        assert torch.equal(state, kept)
        y2 = rsm.selective_scan_step(*args(t), state, z=zt, **opt)
        assert torch.equal(y, y2) and torch.equal(state, other)
        check("y", f64(y), np.stack([r["y"][t] for r in ref]), np.stack([r["by"][t] for r in ref]))
    check("state", f64(state), np.stack([r["final"] for r in ref]), np.stack([r["bfinal"] for r in ref]))
    # without gate, skip, bias and softplus
    s1 = state.clone()
    y = rsm.selective_scan_step(*args(0), s1, softplus=False)
    x, dt, Bv, Cv = (f64(a[k][:, 0]) for k in ("x", "dt", "B", "C"))
    for i in range(B):
        f = O.ssm(x[i:i + 1], dt[i:i + 1], f64(a["A"]), Bv[i:i + 1], Cv[i:i + 1], softplus=False, init=f64(state)[i])
        size = np.abs(f64(state)[i]) * np.exp(dt[i][:, None] * f64(a["A"])) + np.abs(dt[i] * x[i])[:, None] * np.abs(Bv[i])
        e = size * 8 * (np.abs(dt[i][:, None] * f64(a["A"])) + 4) * U
        check("state", f64(s1)[i], f["final"], e)
        check("y", f64(y)[i], f["y"][0], e @ np.abs(Cv[i]) + (N + 4) * U * (size @ np.abs(Cv[i])) + half(dtype) * np.abs(f["y"][0]))


def test_far_steps():
    """Steps so large that states are forgotten at once, so small that nothing moves, and no steps at all."""
    import torch
    a = inputs(60, (1, 200), 1, 16, 16, "fp32")
    a["dt"][:, 20:40] = 60.0
    a["dt"][:, 60:90] = -60.0
    a["dt"][:, 120:125] = float("-inf")
    a["dt"][:, 150] = 3e4
    y, final, g = run(a, None, True)
    assert all(torch.isfinite(t).all() for t in (y, final, *g.values()))
    a["dt"][:, 120:125] = -200.0          # the same step of 0, but numbers for the bounds
    y2, final2, _ = run(a, None, True)
    assert torch.equal(y, y2) and torch.equal(final, final2)
    a["dt"][:, 150] = 60.0
    compare(a, [200], "fp32", True, run(a, None, True))


def test_sequences_keep_to_themselves():
    import torch
    lens = [70, 9, 0, 2, 300]
    total = sum(lens)
    a = inputs(80, (total + 7,), 5, 40, 16, "bf16")

    def call(a):
        import recurrent_sequence_models_amd as rsm
        opt = dict(D=a["D"], z=a["z"], dt_bias=a["bias"], cu_seqlens=offsets(lens), init=a["init"])
        args = a["x"], a["dt"], a["A"], a["B"], a["C"]
        y, final, states = rsm.selective_scan(*args, chunk_states=True, out=torch.full_like(a["x"], 7.0), **opt)
        out = {"d" + k: torch.full_like(a[k], 7.0) for k in ("x", "dt", "B", "C", "z")}
        g = rsm.selective_scan_bwd(*args, a["dy"], states, d_final=a["d_final"], out=out, **opt)
        return [y, g["dx"], g["ddt"], g["dB"], g["dC"], g["dz"]], [final, g["d_init"]]
    good = call(a)
    for t in good[0]:
        assert torch.all(t[total:] == 7)
    bad = {k: t.clone() for k, t in a.items()}
    for k in NAMES:
        bad[k][70:79], bad[k][total:] = float("nan"), float("inf")
    bad["init"][1], bad["d_final"][1] = float("inf"), float("nan")
    got = call(bad)
    keep = torch.tensor([i for i in range(total) if not 70 <= i < 79], device="cuda")
    for p, q in zip(got[0], good[0]):
        assert torch.equal(p[keep], q[keep]) and torch.all(p[total:] == 7)
    for p, q in zip(got[1], good[1]):
        assert torch.equal(p[[0, 2, 3, 4]], q[[0, 2, 3, 4]])


def test_graphs_streams_and_determinism():
    import torch
    lens = [500, 0, 91, 300]
    a = inputs(90, (891,), 4, 264, 16, "bf16")
    cu = offsets(lens)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")

    def call(**kw):
        y, final, g = run(a, cu, True, workspace=ws, **kw)
        return [y, final, *g.values()]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    same_in_graph(call)


def test_past_32_bits():
    """Tokens behind 2^31 entries."""
    import torch
    import recurrent_sequence_models_amd as rsm
    D, T, N, last = 8192, (1 << 18) + 40, 16, 60
    a = inputs(100, (1, last), 1, D, N, "bf16", gate=False, state=False)
    big = {}
    for k in ("x", "dt", "B", "C"):
        t = big[k] = torch.zeros(1, T, a[k].shape[-1], dtype=torch.bfloat16, device="cuda")
        t[:, -last:] = a[k]
    opt = dict(D=a["D"], dt_bias=a["bias"])
    args, tail = (big["x"], big["dt"], a["A"], big["B"], big["C"]), (a["x"], a["dt"], a["A"], a["B"], a["C"])
    y, final, states = rsm.selective_scan(*args, chunk_states=True, **opt)
    z, end, kept = rsm.selective_scan(*tail, chunk_states=True, **opt)
    assert not y[:, :-last].any()
    torch.testing.assert_close(y[:, -last:].float(), z.float(), rtol=2 ** -7, atol=1e-5)
    torch.testing.assert_close(final, end, rtol=1e-4, atol=1e-6)
    dy = torch.zeros_like(y)
    dy[:, -last:] = a["dy"]
    g, h = rsm.selective_scan_bwd(*args, dy, states, **opt), rsm.selective_scan_bwd(*tail, a["dy"], kept, **opt)
    for k in ("dx", "ddt", "dB", "dC"):
        # sums over up to 8192 channels: two roundings of bf16 apart, relative to the sums' size
        size = h[k].float().abs().mean()
        assert (g[k][:, -last:].float() - h[k].float()).abs().max() <= 2 ** -7 * h[k].float().abs().max() + 1e-3 * size, k
    torch.testing.assert_close(g["dA"], h["dA"], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("N", [16, 64])
@pytest.mark.parametrize("T", [37, 600])
def test_infinite_last_token(T, N):
    """An infinity of a sequence's last token stays an infinity, and in its own state (backward too), where a tile ends
    behind it."""
    import torch
    import recurrent_sequence_models_amd as rsm
    a = inputs(70, (2, T), 2, 40, N, "fp32", gate=False, extras=False)
    a = {k: v if v is None or k == "A" else v.abs() for k, v in a.items()}
    at, rest = 3, [n for n in range(N) if n != 3]

    def run(**change):
        b = {**a, **change}
        x = [b[k] for k in ("x", "dt", "A", "B", "C")]
        y, final, states = rsm.selective_scan(*x, init=b["init"], chunk_states=True)
        return y, final, rsm.selective_scan_bwd(*x, b["dy"], states, init=b["init"], d_final=b["d_final"])

    inf = {k: a[k].clone() for k in ("B", "C")}
    for v in inf.values():
        v[:, -1, at] = float("inf")
    y, final, g = run()
    yb, fb, gb = run(B=inf["B"])
    assert torch.equal(yb[:, :-1], y[:, :-1]) and torch.isposinf(yb[:, -1]).all()
    assert torch.equal(fb[..., rest], final[..., rest]) and torch.isposinf(fb[..., at]).all()
    for k in ("dB", "d_init"):
        assert torch.equal(gb[k], g[k]), k
    for k in ("dA", "dC"):
        assert torch.equal(gb[k][..., rest], g[k][..., rest]), k
    yc, fc, gc = run(C=inf["C"])
    assert torch.equal(yc[:, :-1], y[:, :-1]) and torch.isposinf(yc[:, -1]).all() and torch.equal(fc, final)
    assert torch.equal(gc["dC"], g["dC"])
    for k in ("dA", "dB", "d_init"):
        assert torch.equal(gc[k][..., rest], g[k][..., rest]), k


@pytest.mark.parametrize("n,T,D,N", [(3, 500, 1536, 16), (4, 300, 1024, 64), (8, 330, 1536, 32)])
def test_sequences_cut_once(n, T, D, N):
    """Gradients where sequences are cut into a long segment and the rest, to fill the last round: those of each sequence by
    itself."""
    import torch
    import recurrent_sequence_models_amd as rsm
    a = inputs(80, (n, T), n, D, N, "bf16")
    opt = lambda i: dict(D=a["D"], z=a["z"][i], dt_bias=a["bias"], init=a["init"][i])  # noqa: E731

    def grads(i):
        x = [a[k][i] for k in ("x", "dt")] + [a["A"]] + [a[k][i] for k in ("B", "C")]
        _, _, states = rsm.selective_scan(*x, chunk_states=True, **opt(i))
        return rsm.selective_scan_bwd(*x, a["dy"][i], states, d_final=a["d_final"][i], **opt(i))

    g, each = grads(slice(None)), [grads(slice(i, i + 1)) for i in range(n)]
    for k in ("dx", "ddt", "dB", "dC", "dz", "d_init"):
        want = torch.cat([e[k] for e in each])
        step = 2 ** -8 if want.dtype is torch.bfloat16 else 0.0       # each is rounded once, on either side of a border
        assert ((g[k] - want).float().abs() <= 2 * step * want.float().abs() + 1e-4 * want.float().abs().max()).all(), k
    for k in ("dA", "dD", "ddt_bias"):
        want = sum(e[k] for e in each)
        assert (g[k] - want).abs().max() <= 1e-4 * want.abs().max(), k
