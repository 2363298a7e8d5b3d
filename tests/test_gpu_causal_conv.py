"""GPU tests of the short causal convolution, forward, backward and for single tokens,
elementwise against the fp64 definition.

Bounds, with u = 2^-24: the pre-activation p is off by (taps + 2) u A, A the sum of its terms'
absolute values; silu has a slope of at most 1.1 and silu' one of at most 1/2; the hardware's exp2
and reciprocal give a sigmoid that is off by (2 |p| + 8) u relative; sums over tokens add u a step
(runs, workgroups and their sum: far fewer steps in a row than tokens); results are rounded once."""

import numpy as np
import pytest

from block_helpers import TINY, U, check, f64, half, offsets, rand, same_in_graph, split, strided, tdt
from oracle import block as O

pytestmark = pytest.mark.gpu

LENS = [[1], [5], [2, 1, 3], [0, 4, 0, 0, 1, 70, 0], [300, 1, 33], [700], [1] * 40, [16, 16, 64, 3, 61]]


def conv_bounds(x, w, b, init, act, dtype, dy=None, d_final=None):
    """dict of values and bounds of one sequence."""
    W = w.shape[1]
    y, final, p = O.conv(x, w, b, init, act)
    A = O.conv(np.abs(x), np.abs(w), np.abs(b), np.abs(init))[2]
    ep = (W + 2) * U * A
    out = dict(y=y, final=final, by=1.1 * ep + np.abs(y) * (2 * np.abs(p) + 10) * U + half(dtype) * np.abs(y) + TINY * (1 + np.abs(p)))
    if dy is not None:
        g = O.conv_backward(x, w, b, init, dy, d_final, act)
        ed = np.abs(dy) * (0.5 * ep + 16 * U * (1 + np.abs(p)) if act else 0 * p) + U * np.abs(g["d"])
        back = O.conv_backward(np.abs(x), np.abs(w), b, np.abs(init), ed, 0 * d_final)     # errors through the same sums
        size = O.conv_backward(np.abs(x), np.abs(w), b, np.abs(init), np.abs(g["d"]), np.abs(d_final))
        out.update(g)
        for n in ("dx", "dinit"):
            out["b" + n] = back[n] + (W + 2) * U * size[n] + half(dtype) * np.abs(g[n]) + TINY
        for n in ("dw", "db"):
            out["b" + n] = back[n] + (min(x.shape[0], 64) + 100) * U * size[n] + TINY
    return out


def both(call, dtype, lens, D, taps, act, init, dense=False, view=False, seed=1):
    """Inputs, and what the sequences give one by one."""
    import torch
    n, total = len(lens), sum(lens)
    lead = (n, lens[0]) if dense else (total,)
    x, dy = rand(seed, *lead, D, dtype=dtype), rand(seed + 1, *lead, D, dtype=dtype)
    w, b = rand(seed + 2, D, taps, scale=0.6), rand(seed + 3, D, scale=0.3)
    s0 = rand(seed + 4, n, taps - 1, D, dtype=dtype) if init else None
    df = rand(seed + 5, n, taps - 1, D, dtype=dtype) if init else None
    cu = None if dense else offsets(lens)
    xv = strided(x) if view else x
    y, fin, g = call(xv, w, b, s0, df, dy, cu)
    torch.cuda.synchronize()
    zero = np.zeros((n, taps - 1, D))
    S, F = (f64(s0), f64(df)) if init else (zero, zero)
    want = [conv_bounds(a, f64(w), f64(b), s, act, dtype, h, f)
            for a, h, s, f in zip(split(f64(x).reshape(-1, D), lens), split(f64(dy).reshape(-1, D), lens), S, F)]
    cat = lambda name: np.concatenate([r[name] for r in want])      # noqa: E731
    check("y", f64(y).reshape(-1, D), cat("y"), cat("by"))
    assert np.array_equal(f64(fin), np.stack([r["final"] for r in want]))
    check("dx", f64(g["dx"]).reshape(-1, D), cat("dx"), cat("bdx"))
    check("d_init", f64(g["d_init"]), np.stack([r["dinit"] for r in want]), np.stack([r["bdinit"] for r in want]))
    # sums over the sequences: their own, and one rounding a sequence
    for name, key in (("dweight", "dw"), ("dbias", "db")):
        check(name, f64(g[name]), sum(r[key] for r in want),
              sum(r["b" + key] for r in want) + (n + 4) * U * sum(np.abs(r[key]) for r in want))


def calls(act, view=False):
    import recurrent_sequence_models_amd as rsm

    def call(x, w, b, s0, df, dy, cu):
        import torch
        kw = dict(bias=b, activation=act, cu_seqlens=cu, init=s0)
        y, fin = rsm.causal_conv(x, w, **kw)
        out = strided(torch.empty(x.shape, dtype=x.dtype, device="cuda")) if view else None
        return y, fin, rsm.causal_conv_bwd(x, w, dy, d_final=df, out=out, **kw)
    return call


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:7])))
@pytest.mark.parametrize("dtype,taps,act", [("bf16", 4, "silu"), ("fp32", 4, None), ("bf16", 3, None), ("fp32", 2, "silu"),
                                            ("fp32", 3, "silu"), ("bf16", 2, "silu")])
def test_packed(dtype, lens, taps, act):
    both(calls(act), dtype, lens, 136, taps, act, init=True)


@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (3, 2, 64), (2, 65, 264), (5, 100, 1536), (40, 7, 128)])
@pytest.mark.parametrize("dtype,init,view", [("bf16", False, False), ("fp32", True, True), ("bf16", True, True)])
def test_batch(dtype, B, T, D, init, view):
    both(calls("silu", view), dtype, [T] * B, D, 4, "silu", init, dense=True, view=view)


@pytest.mark.parametrize("run", [8, 16])
def test_longer_runs(run):
    """Sizes at which threads own runs of 8 and of 16 tokens."""
    D = 4096 if run == 16 else 1536
    lens = [777, 0, 1, 2300 - 778] if run == 16 else [1000, 3, 2000]
    both(calls("silu"), "bf16", lens, D, 4, "silu", init=True)


def test_without_bias():
    import torch
    import recurrent_sequence_models_amd as rsm
    x, w, dy = rand(1, 2, 30, 64), rand(2, 64, 4), rand(3, 2, 30, 64)
    zero = torch.zeros(64, device="cuda")
    y, _ = rsm.causal_conv(x, w, final=False)
    z, _ = rsm.causal_conv(x, w, bias=zero)
    assert torch.equal(y, z)
    a, b = rsm.causal_conv_bwd(x, w, dy, d_init=False), rsm.causal_conv_bwd(x, w, dy, bias=zero)
    assert a["dbias"] is None and a["d_init"] is None
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])


def test_gradients_are_those_of_differences():
    r = np.random.default_rng(5)
    x, w, b, s, dy, df = (r.normal(size=n) for n in ((6, 4), (4, 3), 4, (2, 4), (6, 4), (2, 4)))
    g = O.conv_backward(x, w, b, s, dy, df, "silu")

    def f(x, w, b, s):
        y, fin, _ = O.conv(x, w, b, s, "silu")
        return (dy * y).sum() + (df * fin).sum()
    args = [x, w, b, s]
    for i, name in enumerate(("dx", "dw", "db", "dinit")):
        d, h = r.normal(size=args[i].shape), 1e-6
        up, down = ([a + t * d if j == i else a for j, a in enumerate(args)] for t in (h, -h))
        assert abs((f(*up) - f(*down)) / (2 * h) - (g[name] * d).sum()) < 1e-7, name


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("taps", [2, 3, 4])
def test_single_tokens_continue_a_prompt(dtype, taps):
    """The bits of the whole sequence's outputs and states, in place and into another state."""
    import torch
    import recurrent_sequence_models_amd as rsm
    B, T, D = 3, 9, 72
    x, w, b = rand(1, B, T, D, dtype=dtype), rand(2, D, taps), rand(3, D)
    kw = dict(bias=b, activation="silu")
    y, fin = rsm.causal_conv(x, w, **kw)
    _, state = rsm.causal_conv(x[:, :4].contiguous(), w, **kw)
    for t in range(4, T):
        xt = strided(x[:, t].contiguous())
        other = torch.empty_like(state)
        kept = state.clone()
        a = rsm.causal_conv_step(xt, w, state, state_out=other, **kw)
        assert torch.equal(state, kept)
        b2 = rsm.causal_conv_step(xt, w, state, **kw)
        assert torch.equal(a, b2) and torch.equal(other, state) and torch.equal(a, y[:, t])
    assert torch.equal(state, fin)


def test_sequences_keep_to_themselves():
    """No numbers in one sequence, and tokens behind the last one."""
    import torch
    import recurrent_sequence_models_amd as rsm
    lens, D = [20, 7, 0, 2, 30], 64
    total = sum(lens)
    x, dy, w = rand(1, total + 9, D, dtype="bf16"), rand(2, total + 9, D, dtype="bf16"), rand(3, D, 4)
    s0, df = rand(4, 5, 3, D, dtype="bf16"), rand(5, 5, 3, D, dtype="bf16")
    cu = offsets(lens)

    def call(x, s0, df, dy):
        out, dx = (torch.full_like(x, 7.0) for _ in range(2))
        y, fin = rsm.causal_conv(x, w, activation="silu", cu_seqlens=cu, init=s0, out=out)
        g = rsm.causal_conv_bwd(x, w, dy, activation="silu", cu_seqlens=cu, init=s0, d_final=df, out=dx)
        return y, g["dx"], fin, g["d_init"]
    good = call(x, s0, df, dy)
    assert torch.all(good[0][total:] == 7) and torch.all(good[1][total:] == 7)
    bad = [t.clone() for t in (x, s0, df, dy)]
    bad[0][20:27], bad[1][1], bad[2][1], bad[3][20:27] = float("nan"), float("inf"), float("nan"), float("inf")
    bad[0][total:], bad[3][total:] = float("nan"), float("nan")
    got = call(*bad)
    keep = torch.tensor([i for i in range(total) if not 20 <= i < 27], device="cuda")
    for a, b in zip(got[:2], good[:2]):
        assert torch.equal(a[keep], b[keep])
    for a, b in zip(got[2:], good[2:]):
        assert torch.equal(a[[0, 2, 3, 4]], b[[0, 2, 3, 4]])


def test_graphs_streams_and_determinism():
    import torch
    import recurrent_sequence_models_amd as rsm
    lens, D = [200, 0, 91], 264
    x, dy = rand(1, 291, D, dtype="bf16"), rand(2, 291, D, dtype="bf16")
    w, b, s0, df = rand(3, D, 4), rand(4, D), rand(5, 3, 3, D, dtype="bf16"), rand(6, 3, 3, D, dtype="bf16")
    cu = offsets(lens)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def call(stream=None):
        kw = dict(bias=b, activation="silu", cu_seqlens=cu, init=s0, stream=stream)
        y, fin = rsm.causal_conv(x, w, **kw)
        g = rsm.causal_conv_bwd(x, w, dy, d_final=df, workspace=ws, **kw)
        return [y, fin, g["dx"], g["dweight"], g["dbias"], g["d_init"]]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    same_in_graph(call)


def test_past_32_bits():
    """Tokens behind 2^31 entries, and a token stride."""
    import torch
    import recurrent_sequence_models_amd as rsm
    D, T = 8192, (1 << 18) + 40
    x = torch.zeros(1, T, D, dtype=torch.bfloat16, device="cuda")
    tail = rand(1, 1, 60, D, dtype="bf16")
    x[:, -60:] = tail
    w = rand(2, D, 4)
    y, fin = rsm.causal_conv(x, w)
    z, end = rsm.causal_conv(tail, w)
    assert torch.equal(y[:, -60:], z) and torch.equal(fin, end) and not y[:, :-60].any()
    g = rsm.causal_conv_bwd(x, w, y, d_init=False, out=y.clone())
    h = rsm.causal_conv_bwd(tail, w, z, d_init=False)
    assert torch.equal(g["dx"][:, -60:], h["dx"])
    torch.testing.assert_close(g["dweight"], h["dweight"], rtol=1e-4, atol=1e-4)
