"""GPU runs of the layer operators together, as a stack uses them: one projection's output
through the query / key norm with rotary positions into the mixers (Falcon, causal
attention) and back, beside the gated recurrence; prompts continued by single tokens.

Compared with the fp64 oracles by the relative L2 bar of the parity tests (gpu_helpers.TOL),
as each stage rounds its results once."""

import numpy as np
import pytest

import oracle
from gpu_helpers import TOL, rel_l2
from layer_helpers import f64, offsets, rand
from oracle import layer as L

pytestmark = pytest.mark.gpu

CASES = [("bf16", [37, 1, 90, 64]), ("fp32", [50, 33])]


def bar(dtype, got, want):
    for n in want:
        e = rel_l2(f64(got[n]), want[n])
        assert np.all(np.isfinite(f64(got[n]))) and e <= TOL[dtype], (n, e)


@pytest.mark.parametrize("dtype,lens", CASES)
def test_attention_layer(dtype, lens):
    """Packed prompts: norm, rotation, attention, a gated recurrence over its output, and all
    gradients back into one gradient of the projection's output."""
    import torch
    import recurrent_sequence_models_amd as rsm
    hq, hk, d, total = 4, 2, 64, sum(lens)
    qkv = rand(1, total, hq + 2 * hk, d, dtype=dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    wq, wk = 1 + 0.2 * rand(2, d), 1 + 0.2 * rand(3, d)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    freq, scale = rsm.rope_frequencies(32, 500000.0, scaling="parts", factor=4.0, original_length=64, device="cuda")
    g = -0.2 * torch.rand(total, hq * d, generator=torch.Generator().manual_seed(1)).cuda().to(qkv.dtype)
    dh = rand(5, total, hq * d, dtype=dtype)
    cu = offsets(lens)
    kw = dict(q_weight=wq, k_weight=wk, rot_scale=scale)
    yq, yk = rsm.qk_norm_rope(q, k, pos, freq, **kw)
    o, lse = rsm.attention_fwd(yq, yk, v, cu_seqlens=cu)
    x = o.view(total, hq * d)
    h, fin, st = rsm.gated_scan(x, g, cu_seqlens=cu, mix=True, chunk_states=True)
    gs = rsm.gated_scan_bwd(x, g, dh, st, cu_seqlens=cu, mix=True)
    grad = torch.empty_like(qkv)
    ga = rsm.attention_bwd(yq, yk, v, o, lse, gs["dx"].view_as(o), cu_seqlens=cu,
                           out=dict(dq=torch.empty_like(yq), dk=torch.empty_like(yk), dv=grad[:, hq + hk:]))
    gq = rsm.qk_norm_rope_bwd(q, k, pos, freq, ga["dq"], ga["dk"], out=dict(dq=grad[:, :hq], dk=grad[:, hq:hq + hk]), **kw)
    torch.cuda.synchronize()

    Q, K, V, G, DH, P, F = (f64(t) for t in (q, k, v, g, dh, pos, freq))
    okw = dict(scale=scale)
    oq, ok = L.norm_rope(Q, f64(wq), P, F, **okw), L.norm_rope(K, f64(wk), P, F, **okw)
    want = {n: np.zeros_like(a) for n, a in (("h", DH), ("dx", DH), ("dg", DH), ("dyq", Q), ("dyk", K), ("dv", V))}
    for a, b in L.ranges(lens):
        f = L.attention(oq[a:b], ok[a:b], V[a:b])
        X = f["o"].reshape(b - a, -1)
        want["h"][a:b], _ = L.gated_scan(X, G[a:b], None, True)
        r = L.gated_scan_backward(X, G[a:b], DH[a:b], None, None, True)
        want["dx"][a:b], want["dg"][a:b] = r["dx"], r["dg"]
        r = L.attention_backward(oq[a:b], ok[a:b], V[a:b], r["dx"].reshape(f["o"].shape))
        want["dyq"][a:b], want["dyk"][a:b], want["dv"][a:b] = r["dq"], r["dk"], r["dv"]
    dq, dwq = L.norm_rope_backward(Q, f64(wq), P, F, want["dyq"], **okw)
    dk, dwk = L.norm_rope_backward(K, f64(wk), P, F, want["dyk"], **okw)
    bar(dtype, dict(h=h, dx=gs["dx"], dg=gs["dg"], grad=grad, dwq=gq["dq_weight"], dwk=gq["dk_weight"]),
        dict(h=want["h"], dx=want["dx"], dg=want["dg"], grad=np.concatenate([dq, dk, want["dv"]], 1), dwq=dwq, dwk=dwk))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_falcon_layer(dtype):
    """Norm and rotation before Falcon: its single-precision gradients go back through them."""
    import torch
    import recurrent_sequence_models_amd as rsm
    B, T, H, d, chunk = 2, 100, 3, 64, 32
    q, k, v = (rand(i, B, T, H, d, dtype=dtype) for i in (1, 2, 3))
    beta, lam = torch.sigmoid(rand(4, B, T, H)), -0.1 * torch.rand(B, T, H, generator=torch.Generator().manual_seed(2)).cuda()
    w = 1 + 0.2 * rand(5, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    freq, _ = rsm.rope_frequencies(64, device="cuda")
    do = rand(6, B, T, H, d, dtype=dtype)
    yq, yk = rsm.qk_norm_rope(q, k, pos, freq, q_weight=w, k_weight=w, layout="interleaved")
    o, _, cs = rsm.chunk_fwd("F1", yq, yk, v, beta, lam, chunk=chunk, chunk_states=True)
    gf = rsm.chunk_bwd("F1", yq, yk, v, beta, lam, do, cs, chunk=chunk)
    gq = rsm.qk_norm_rope_bwd(q, k, pos, freq, gf["dq"], gf["dk"], q_weight=w, k_weight=w, layout="interleaved")
    torch.cuda.synchronize()
    assert gf["dq"].dtype == torch.float32 and gq["dq"].dtype == q.dtype
    flat = lambda t: f64(t).reshape(B * T, H, d)  # noqa: E731
    P, F, W = f64(pos).reshape(-1), f64(freq), f64(w)
    oq = L.norm_rope(flat(q), W, P, F, layout="interleaved").reshape(B, T, H, d)
    ok = L.norm_rope(flat(k), W, P, F, layout="interleaved").reshape(B, T, H, d)
    args = dict(q=oq, k=ok, v=f64(v), beta=f64(beta), log_lambda=f64(lam))
    ref = oracle.recurrent("F1", **args)
    r = oracle.recurrent_backward("F1", **args, do=f64(do))
    dq, dwq = L.norm_rope_backward(flat(q), W, P, F, r["dq"].reshape(B * T, H, d), layout="interleaved")
    dk, dwk = L.norm_rope_backward(flat(k), W, P, F, r["dk"].reshape(B * T, H, d), layout="interleaved")
    bar(dtype, dict(o=o, dq=gq["dq"].view(B * T, H, d), dk=gq["dk"].view(B * T, H, d), dwq=gq["dq_weight"],
                    dwk=gq["dk_weight"]), dict(o=ref["o"], dq=dq, dk=dk, dwq=dwq, dwk=dwk))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_single_tokens_continue_a_prompt(dtype):
    """Tokens one at a time against the keys and values kept so far give what the whole
    prompt gives."""
    import torch
    import recurrent_sequence_models_amd as rsm
    hq, hk, d, lens, more = 4, 2, 64, [70, 3, 300], 3
    freq, _ = rsm.rope_frequencies(64, device="cuda")
    seqs = [rand(10 + i, n + more, hq + 2 * hk, d, dtype=dtype) for i, n in enumerate(lens)]
    cut = lambda t: (t[:, :hq], t[:, hq:hq + hk], t[:, hq + hk:])  # noqa: E731
    at = lambda ts: torch.cat([torch.as_tensor(t) for t in ts]).int().cuda()  # noqa: E731
    # the whole sequences at once
    q, k, v = cut(torch.cat(seqs))
    yq, yk = rsm.qk_norm_rope(q, k, at([torch.arange(n + more) for n in lens]), freq)
    whole, _ = rsm.attention_fwd(yq, yk, v, cu_seqlens=offsets([n + more for n in lens]))
    ends = np.cumsum([n + more for n in lens])
    # the prompts, then a token a call
    kept = []
    for s, n in zip(seqs, lens):
        _, k, v = cut(s[:n])
        kept.append([rsm.qk_norm_rope(s[:n, :hq], k, torch.arange(n, dtype=torch.int32, device="cuda"), freq)[1], v])
    for t in range(more):
        q, k, v = cut(torch.stack([s[n + t] for s, n in zip(seqs, lens)]))
        yq, yk = rsm.qk_norm_rope(q, k, torch.tensor([n + t for n in lens], dtype=torch.int32, device="cuda"), freq)
        for i, kv in enumerate(kept):
            kv[0], kv[1] = torch.cat([kv[0], yk[i:i + 1]]), torch.cat([kv[1], v[i:i + 1]])
        o, _ = rsm.attention_fwd(yq, torch.cat([kv[0] for kv in kept]), torch.cat([kv[1] for kv in kept]),
                                 cu_seqlens=offsets([1] * len(lens)), cu_seqlens_k=offsets([n + t + 1 for n in lens]))
        for i in range(len(lens)):
            want = f64(whole[int(ends[i]) - more + t])
            assert rel_l2(f64(o[i]), want) <= TOL[dtype] / 2, (t, i)


def test_graphs_that_share_a_workspace():
    """Two captured graphs whose calls were given the same workspaces, replayed in turn with eager
    calls on them between."""
    import torch
    from recurrent_sequence_models_amd import (attention_bwd, attention_fwd, gated_scan, gated_scan_bwd, qk_norm_rope_bwd,
                                               rope_frequencies)
    x, g, dh = (rand(i, 2, 1500, 72, dtype="bf16") for i in (1, 2, 3))
    g = -g.abs()
    q, k, v, do = (rand(i, 700, h, 64, dtype="bf16") for i, h in ((4, 4), (5, 2), (6, 2), (7, 4)))
    one, cu, cuk = rand(8, 1, 4, 64, dtype="bf16"), offsets([1]), offsets([700])
    pos, freq = torch.arange(700, dtype=torch.int32, device="cuda"), rope_frequencies(64, device="cuda")[0]
    w = rand(9, 64)
    ws = [torch.empty(1 << 24, dtype=torch.uint8, device="cuda") for _ in range(4)]

    def call(sign):
        h, _, st = gated_scan(x, g, mix=sign, chunk_states=True, workspace=ws[0])
        b = gated_scan_bwd(x, g, dh, st, mix=sign, workspace=ws[0])
        o, lse = attention_fwd(q, k, v, scale=0.1 + 0.1 * sign, cu_seqlens=cuk, workspace=ws[1])
        t, _ = attention_fwd(one, k, v, scale=0.1 + 0.1 * sign, cu_seqlens=cu, cu_seqlens_k=cuk, workspace=ws[1])
        a = attention_bwd(q, k, v, o, lse, do, scale=0.1 + 0.1 * sign, cu_seqlens=cuk, workspace=ws[2])
        n = qk_norm_rope_bwd(q, k, pos, freq, do, k, q_weight=w, k_weight=w, rot_scale=1.0 + sign, workspace=ws[3])
        return [h, st, *b.values(), o, t, *a.values(), *n.values()]

    want = [call(False), call(True)]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], [None, None]
    for i in (0, 1):
        with torch.cuda.graph(graphs[i]):
            got[i] = call(bool(i))
    for turn in (0, 1, 1, 0, 1):
        for t in got[turn]:
            t.zero_()
        graphs[turn].replay()
        eager = call(not turn)
        torch.cuda.synchronize()
        for a, b, c, d in zip(got[turn], want[turn], eager, want[not turn]):
            assert torch.equal(a, b) and torch.equal(c, d)
