"""GPU parity of the gated linear recurrence (falcon_scan_fwd, _bwd, _step) against the
fp64 oracle, elementwise, with bounds derived in layer_helpers."""

import numpy as np
import pytest

from layer_helpers import SCAN_C, U, check, f64, half, offsets, rand, scan_back_bounds, scan_bounds
from oracle import layer as L

pytestmark = pytest.mark.gpu


def gates(seed, *shape, dtype, kind="slow"):
    """Log decays: near 0 ("slow"), spread widely with exact resets ("mixed")."""
    import torch
    r = np.random.Generator(np.random.PCG64(seed))
    g = -np.log1p(np.exp(r.normal(size=shape))) * 0.1
    if kind == "mixed":
        g = -np.exp(r.uniform(np.log(1e-4), np.log(30.0), size=shape))
        g[r.random(shape) < 0.02] = -np.inf
        g[r.random(shape) < 0.02] = 0.0
    t = torch.from_numpy(g.astype(np.float32))
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


def sequences(x, cu_lens):
    """Index of every sequence in the token axes: (row or None, begin, end)."""
    if cu_lens is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    return [(None, a, b) for a, b in L.ranges(cu_lens)]


def part(a, row, lo, hi):
    return a[lo:hi] if row is None else a[row, lo:hi]


def run_case(dtype, shape, mix, lens=None, init=True, kind="slow", seed=1, back=True, behind=0):
    """Forward and backward of one batch, every sequence against the oracle."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_bwd
    if lens is not None:
        shape = (sum(lens) + behind, shape[-1])
    n, D = (len(lens) if lens is not None else shape[0]), shape[-1]
    x, dh = rand(seed, *shape, dtype=dtype), rand(seed + 1, *shape, dtype=dtype)
    g = gates(seed + 2, *shape, dtype=dtype, kind=kind)
    h0 = rand(seed + 3, n, D) if init else None
    df = rand(seed + 4, n, D)
    cu = offsets(lens) if lens is not None else None
    out = torch.full_like(x, 7.0)
    h, fin, states = gated_scan(x, g, cu_seqlens=cu, mix=mix, init=h0, chunk_states=True, out=out)
    gr = gated_scan_bwd(x, g, dh, states, cu_seqlens=cu, mix=mix, init=h0, d_final=df,
                        out=dict(dx=torch.full_like(x, 7.0), dg=torch.full_like(x, 7.0)))
    torch.cuda.synchronize()
    X, G, DH, H0, DF = f64(x), f64(g), f64(dh), f64(h0), f64(df)
    h, fin = f64(h), f64(fin)
    gr = {k: f64(v) for k, v in gr.items()}
    for i, (row, lo, hi) in enumerate(sequences(X, lens)):
        xs, gs, ds = part(X, row, lo, hi), part(G, row, lo, hi), part(DH, row, lo, hi)
        hi0 = H0[i] if init else None
        if hi == lo:       # an empty sequence: its end is its beginning
            assert np.array_equal(fin[i], hi0 if init else np.zeros(D))
            assert np.array_equal(gr["d_init"][i], DF[i])
            continue
        ref, rfin = L.gated_scan(xs, gs, hi0, mix)
        H, E = scan_bounds(xs, gs, hi0, mix)
        check(f"h[{i}]", part(h, row, lo, hi), ref, half(dtype) * np.abs(ref) * (1 + 1e-3) + E)
        check(f"final[{i}]", fin[i], rfin, E[-1] + U * np.abs(rfin))
        if not back:
            continue
        want = L.gated_scan_backward(xs, gs, ds, DF[i], hi0, mix)
        er, Dabs, lam = scan_back_bounds(xs, gs, ds, DF[i], hi0, mix)
        w = 1 - lam if mix else np.ones_like(lam)
        check(f"dx[{i}]", part(gr["dx"], row, lo, hi), want["dx"],
              half(dtype) * np.abs(want["dx"]) * (1 + 1e-3) + w * (er + SCAN_C * U * Dabs))
        prev = np.vstack([np.zeros((1, D)) if hi0 is None else hi0[None], ref[:-1]])
        eprev = np.vstack([np.zeros((1, D)), E[:-1]])
        inner = prev - xs if mix else prev
        bound = lam * (er + SCAN_C * U * Dabs) * np.abs(inner) + lam * Dabs * (eprev + U * (np.abs(prev) + np.abs(xs)))
        check(f"dg[{i}]", part(gr["dg"], row, lo, hi), want["dg"],
              half(dtype) * np.abs(want["dg"]) * (1 + 1e-3) + bound * (1 + 1e-3))
        check(f"d_init[{i}]", gr["d_init"][i], want["d_init"], lam[0] * (er[0] + SCAN_C * U * Dabs[0]))
    if behind:             # tokens behind the last sequence are left as they were
        for a in (f64(out), gr["dx"], gr["dg"]):
            assert np.all(a[-behind:] == 7.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 255, 256, 257, 700])
def test_batch(dtype, mix, T):
    run_case(dtype, (3, T, 72), mix, seed=T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [8, 56, 64, 136, 768])
def test_widths(dtype, D):
    run_case(dtype, (2, 300, D), True, seed=D)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mix", [False, True])
def test_wide_decays_and_resets(dtype, mix):
    """Decays from 1 down to e^-30 and exact zeros."""
    run_case(dtype, (2, 600, 64), mix, kind="mixed", seed=5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [4096, 8192 + 5])
def test_long(dtype, T):
    """Several groups of chunks: carries pass through the published group states."""
    run_case(dtype, (1, T, 16), True, seed=T, kind="slow")


PACKED = [[1], [5, 0, 0, 3], [1] * 40, [3, 1, 1, 2, 900, 1, 0, 255, 256, 1, 257], [0, 0, 17, 0], [2000, 3000, 50],
          [256, 256, 256], [4, 4, 8, 8, 1, 7, 16]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", PACKED, ids=lambda p: "-".join(map(str, p[:6])))
@pytest.mark.parametrize("mix,init", [(False, True), (True, False)])
def test_packed(dtype, lens, mix, init):
    run_case(dtype, (sum(lens), 40), mix, lens=lens, init=init, seed=len(lens))


@pytest.mark.parametrize("n", [62, 63, 64, 65, 400, 4200])
def test_many_sequences(n):
    """More sequences than one register of offsets holds, and more than 64 x 64; some empty."""
    r = np.random.Generator(np.random.PCG64(n))
    run_case("fp32", (0, 8), True, lens=[int(x) for x in r.integers(0, 9 if n < 1000 else 3, size=n)], seed=n)


@pytest.mark.parametrize("behind", [1, 300])
def test_packed_leaves_the_rest(behind):
    """Tokens behind the last sequence are not written, nor is anything read as theirs."""
    run_case("bf16", (600 + behind, 64), False, lens=[100, 0, 500], behind=behind)


def test_one_sequence_does_not_reach_the_next():
    """NaN and infinities of one packed sequence stay in it, in both directions."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_bwd
    lens, D = [300, 310, 5], 64
    x, dh = rand(1, 615, D), rand(2, 615, D)
    g = gates(3, 615, D, dtype="fp32")
    cu = offsets(lens)
    bad, dbad = x.clone(), dh.clone()
    bad[290, ::2], bad[290, 1::2] = float("nan"), float("inf")
    dbad[320, ::2], dbad[320, 1::2] = float("nan"), float("inf")
    h, fin, st = gated_scan(x, g, cu_seqlens=cu, chunk_states=True)
    h2, fin2, st2 = gated_scan(bad, g, cu_seqlens=cu, chunk_states=True)
    assert torch.equal(h[300:], h2[300:]) and torch.equal(fin[1:], fin2[1:])
    assert not torch.isfinite(h2[290:300]).any()
    a = gated_scan_bwd(x, g, dh, st, cu_seqlens=cu)
    b = gated_scan_bwd(x, g, dbad, st, cu_seqlens=cu)
    for n in ("dx", "dg"):
        assert torch.equal(a[n][:300], b[n][:300]) and torch.equal(a[n][610:], b[n][610:])
    assert not torch.isfinite(b["dx"][300:321]).any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[40, 8, 252, 4, 4, 192, 300], [20, 12, 12, 12, 12, 700, 12, 12, 300, 9, 9],
                                  [300] + [5] * 130 + [600]], ids=["few", "waves", "many"])
def test_several_starts_behind_a_nonfinite_sequence(dtype, lens):
    """However many sequences begin in a stretch of steps, none of them sees what is before the
    stretch (forward) or behind it (backward)."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_bwd
    T, D, cu = sum(lens), 64, offsets(lens)
    first, last = lens[0], T - lens[-1]
    x, dh = rand(41, T, D, dtype=dtype), rand(42, T, D, dtype=dtype)
    g = gates(43, T, D, dtype=dtype)
    bad, dbad = x.clone(), dh.clone()
    bad[:first, ::2], bad[:first, 1::2] = float("nan"), float("inf")
    dbad[last:, ::2], dbad[last:, 1::2] = float("nan"), float("inf")
    h0, fin0, states0 = gated_scan(x, g, cu_seqlens=cu, chunk_states=True)
    h1, fin1, _ = gated_scan(bad, g, cu_seqlens=cu)
    assert torch.equal(h0[first:], h1[first:]) and torch.equal(fin0[1:], fin1[1:])
    assert not h1[:first].isfinite().any() and not fin1[0].isfinite().any()
    r0 = gated_scan_bwd(x, g, dh, states0, cu_seqlens=cu)
    r1 = gated_scan_bwd(x, g, dbad, states0, cu_seqlens=cu)
    for k in ("dx", "dg"):
        assert torch.equal(r0[k][:last], r1[k][:last]), k
    assert torch.equal(r0["d_init"][:-1], r1["d_init"][:-1])
    assert not r1["dx"][last:].isfinite().any()


@pytest.mark.parametrize("packed", [False, True])
def test_in_place_state_and_continuation(packed):
    """final may be init; two halves in a row equal the whole."""
    import torch
    from recurrent_sequence_models_amd import gated_scan
    B, T, D = 3, 1000, 64
    x, g, h0 = rand(1, B, T, D), gates(2, B, T, D, dtype="fp32"), rand(3, B, D)
    if packed:
        lens = [T] * B
        whole, fin, _ = gated_scan(x.view(B * T, D), g.view(B * T, D), cu_seqlens=offsets(lens), init=h0)
        st = h0.clone()
        got, same, _ = gated_scan(x.view(B * T, D), g.view(B * T, D), cu_seqlens=offsets(lens), init=st, final=st)
        assert same is st and torch.equal(whole, got) and torch.equal(st, fin)
        return
    whole, fin, _ = gated_scan(x, g, init=h0)
    st = h0.clone()
    a, _, _ = gated_scan(x[:, :400].contiguous(), g[:, :400].contiguous(), init=st, final=st)
    b, _, _ = gated_scan(x[:, 400:].contiguous(), g[:, 400:].contiguous(), init=st, final=st)
    _, E = scan_bounds(f64(x[0]), f64(g[0]), f64(h0[0]), False)
    check("halves", f64(torch.cat([a, b], 1))[0], f64(whole)[0], 2 * E)
    check("final", f64(st)[0], f64(fin)[0], 2 * E[-1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("B,D", [(1, 8), (3, 72), (64, 2048)])
def test_step(dtype, mix, B, D):
    import torch
    from recurrent_sequence_models_amd import gated_scan_step
    x, g, st = rand(1, B, D, dtype=dtype), gates(2, B, D, dtype=dtype, kind="mixed"), rand(3, B, D)
    s0 = f64(st)
    h = gated_scan_step(x, g, st, mix=mix)
    torch.cuda.synchronize()
    lam = np.exp(f64(g))
    u = (-np.expm1(f64(g)) if mix else 1.0) * f64(x)
    ref = lam * s0 + u
    bound = SCAN_C * U * (lam * np.abs(s0) + np.abs(u))
    check("state", f64(st), ref, bound)
    check("h", f64(h), ref, bound + half(dtype) * np.abs(ref) * (1 + 1e-3))


def test_steps_continue_a_prompt():
    """A packed prompt's final states go on in single tokens as the longer prompt does."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_step
    lens, D = [37, 300, 1], 64
    xs = [rand(10 + i, n + 4, D) for i, n in enumerate(lens)]
    gs = [gates(20 + i, n + 4, D, dtype="fp32") for i, n in enumerate(lens)]
    _, st, _ = gated_scan(torch.cat([a[:n] for a, n in zip(xs, lens)]), torch.cat([a[:n] for a, n in zip(gs, lens)]),
                          cu_seqlens=offsets(lens), mix=True)
    for t in range(4):
        h = gated_scan_step(torch.stack([a[n + t] for a, n in zip(xs, lens)]),
                            torch.stack([a[n + t] for a, n in zip(gs, lens)]), st, mix=True)
        for i, n in enumerate(lens):
            X, G = f64(xs[i])[:n + t + 1], f64(gs[i])[:n + t + 1]
            ref, _ = L.gated_scan(X, G, None, True)
            _, E = scan_bounds(X, G, None, True)
            check(f"step {t} of {i}", f64(h)[i], ref[-1], E[-1] + 2 * U * np.abs(ref[-1]))


def test_two_streams_and_graphs():
    """Calls on two streams at once, and two captured graphs that share one workspace and
    are replayed in turn, give the eager bits."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_bwd
    from recurrent_sequence_models_amd import falcon as F
    import ctypes
    B, T, D = 2, 3000, 64
    xs = [rand(i, B, T, D, dtype="bf16") for i in range(2)]
    gs = [gates(5 + i, B, T, D, dtype="bf16") for i in range(2)]
    dh = rand(9, B, T, D, dtype="bf16")
    eager = []
    for x, g in zip(xs, gs):
        h, f, s = gated_scan(x, g, chunk_states=True)
        eager.append((h, f, s, gated_scan_bwd(x, g, dh, s)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for x, g, st in zip(xs, gs, streams):
            h, f, s = gated_scan(x, g, chunk_states=True, stream=st)
            got.append((h, f, s, gated_scan_bwd(x, g, dh, s, stream=st)))
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[3]["dg"], b[3]["dg"])
    need = F.lib().falcon_scan_workspace(ctypes.byref(F.ScanShape(1, B, T, D, 0)), 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for x, g in zip(xs, gs):
        out, fin = torch.empty_like(x), torch.empty(B, D, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h, f, s = gated_scan(x, g, out=out, final=fin, chunk_states=True, workspace=ws)
            gr = gated_scan_bwd(x, g, dh, s, workspace=ws)
        graphs.append((graph, out, fin, gr))
    for _ in range(4):
        for (graph, out, fin, gr), e in zip(graphs, eager):
            out.zero_(), fin.zero_(), gr["dx"].zero_(), gr["dg"].zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, e[0]) and torch.equal(fin, e[1])
            assert torch.equal(gr["dx"], e[3]["dx"]) and torch.equal(gr["dg"], e[3]["dg"])


def test_refusals():
    """The binding refuses what the kernels cannot take."""
    import torch
    from recurrent_sequence_models_amd import FalconError, gated_scan, gated_scan_bwd, gated_scan_step
    x = rand(1, 2, 16, 64)
    with pytest.raises(TypeError):
        gated_scan(x.half(), x.half())
    with pytest.raises(TypeError):
        gated_scan(x, x.bfloat16())
    with pytest.raises(ValueError):
        gated_scan(x, x[:, :8])
    with pytest.raises(ValueError):
        gated_scan(x.transpose(0, 1), x.transpose(0, 1))
    with pytest.raises(ValueError):
        gated_scan(x, x, init=torch.zeros(3, 64, device="cuda"))
    with pytest.raises(ValueError):
        gated_scan(x, x, cu_seqlens=offsets([16, 16]))        # a packed call takes [total, D]
    with pytest.raises(TypeError):
        gated_scan(x[0], x[0], cu_seqlens=offsets([16]).long())
    with pytest.raises(FalconError):
        gated_scan(x[..., :60].contiguous(), x[..., :60].contiguous())   # a width not a multiple of 8
    with pytest.raises(FalconError):
        big = rand(1, 1, 600, 64)
        gated_scan(big, big, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gated_scan_bwd(x, x, x, torch.zeros(2, 2, 64, device="cuda"))
    with pytest.raises(ValueError):
        gated_scan_step(x[:, 0].contiguous(), x[:, 0].contiguous(), torch.zeros(2, 32, device="cuda"))
    with pytest.raises(ValueError):
        gated_scan(x.cpu(), x.cpu())


def test_past_32_bits_of_elements():
    """Arrays of over 2^31 elements: the steps behind that place are as in a short call."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_bwd
    D, T, tail = 2048, (1 << 20) + 512 + 5, 517     # the tail begins with a chunk, and with a reset
    cut = slice(T - tail, T)
    x, g, dh = (torch.zeros(1, T, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    x[:, cut], dh[:, cut] = rand(1, 1, tail, D, dtype="bf16"), rand(2, 1, tail, D, dtype="bf16")
    g[:, cut] = gates(3, 1, tail, D, dtype="bf16")
    g[:, T - tail] = float("-inf")
    h, fin, st = gated_scan(x, g, chunk_states=True)
    b = gated_scan_bwd(x, g, dh, st)
    X, G, DH = (t[:, cut].contiguous() for t in (x, g, dh))
    h2, fin2, st2 = gated_scan(X, G, chunk_states=True)
    b2 = gated_scan_bwd(X, G, DH, st2)
    assert torch.equal(h[:, cut], h2) and torch.equal(fin, fin2) and torch.equal(st[:, -3:], st2)
    assert not h[:, :T - tail].any()
    for n in ("dx", "dg"):
        assert torch.equal(b[n][:, cut], b2[n]) and not b[n][:, :T - tail].any(), n


@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("bits", [0x7fc00000, 0x7fffffff, -1, 0x7f800000])
def test_nonfinite_decay_stays_in_its_sequence(bits, mix):
    """Log decays that are NaN (of any payload: memory of all ones too) or +inf make their own
    sequence's states non-finite, not those of a sequence that begins later in the same chunk and
    goes on into the next ones; and so against time."""
    import torch
    from recurrent_sequence_models_amd import gated_scan, gated_scan_bwd
    lens, D = [100, 700, 90, 600], 64
    T, cu = sum(lens), offsets(lens)
    x, dh, g, init = rand(1, T, D), rand(2, T, D), gates(3, T, D, dtype="fp32"), rand(4, 4, D)
    bad = g.clone()
    bad.view(torch.int32)[50], bad.view(torch.int32)[850] = bits, bits      # sequences 0 and 2
    kw = dict(cu_seqlens=cu, mix=mix, init=init)
    h, fin, st = gated_scan(x, g, chunk_states=True, **kw)
    h2, fin2, st2 = gated_scan(x, bad, chunk_states=True, **kw)
    a, b = gated_scan_bwd(x, g, dh, st, **kw), gated_scan_bwd(x, bad, dh, st2, **kw)
    for n, (lo, hi) in enumerate(L.ranges(lens)):
        if n % 2:
            assert torch.equal(h[lo:hi], h2[lo:hi]) and torch.equal(fin[n], fin2[n]), n
            for k in ("dx", "dg"):
                assert torch.equal(a[k][lo:hi], b[k][lo:hi]), (k, n)
            assert torch.equal(a["d_init"][n], b["d_init"][n]), n
        else:
            at = 50 if n == 0 else 850
            assert not h2[at:hi].isfinite().any() and not fin2[n].isfinite().any()
            assert not b["dx"][lo:at].isfinite().any() and not b["d_init"][n].isfinite().any()
