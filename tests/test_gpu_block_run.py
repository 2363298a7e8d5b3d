"""GPU runs of a state-space block's operators together, as a model uses them: the norm of the
stream, the projection into the block, convolution, scan, gate and the projection back to the stream;
training with all gradients, prompts on 8-bit operands, and single tokens that continue them.

Compared with the fp64 oracles by the relative L2 bar of the parity tests (gpu_helpers.TOL), as each
stage rounds its results once."""

import numpy as np
import pytest

from block_helpers import f64, offsets, rand, split
from gpu_helpers import TOL, rel_l2
from oracle import block as O

pytestmark = pytest.mark.gpu


def weights(d, inner, N, R, dtype, seed=1):
    """A block's parameters: two projections in and out, of dt, B and C, the convolution's and the scan's."""
    import torch
    w = dict(norm=1 + 0.2 * rand(seed, d), w_in=rand(seed + 1, 2 * inner, d, dtype=dtype, scale=d ** -0.5),
             conv_w=rand(seed + 2, inner, 4, scale=0.5), conv_b=rand(seed + 3, inner, scale=0.1),
             w_x=rand(seed + 4, R + 2 * N, inner, dtype=dtype, scale=inner ** -0.5), w_dt=rand(seed + 5, inner, R, dtype=dtype, scale=R ** -0.5),
             b_dt=rand(seed + 6, inner, scale=0.5) - 3, D=rand(seed + 7, inner), w_out=rand(seed + 8, d, inner, dtype=dtype, scale=inner ** -0.5))
    w["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * rand(seed + 9, inner, N))
    return w


def block(rsm, w, stream, x, cu, R, N, init=None, bits=False, train=False):
    """x joins the stream, and the block's output is returned beside the new stream (tokens packed)."""
    inner = w["conv_w"].shape[0]
    k = dict(cu_seqlens=cu)
    conv0, ssm0 = init or (None, None)
    if bits:
        u, s, scale = rsm.rms_norm(x, w["norm"], residual=stream, quantize=True)
        q, qs = rsm.quantize_rows(w["w_in"])
        xz, _ = rsm.linear(u, q, x_scale=scale, weight_scale=qs, out_dtype=x.dtype)
    else:
        u, s, _ = rsm.rms_norm(x, w["norm"], residual=stream)
        xz, _ = rsm.linear(u, w["w_in"])
    xs, z = xz[:, :inner], xz[:, inner:]
    c, conv1 = rsm.causal_conv(xs, w["conv_w"], bias=w["conv_b"], activation="silu", init=conv0, **k)
    p, _ = rsm.linear(c, w["w_x"])
    dt, _ = rsm.linear(p[:, :R], w["w_dt"])
    B, C = p[:, R:R + N], p[:, R + N:]
    y, ssm1, states = rsm.selective_scan(c, dt, w["A"], B, C, D=w["D"], z=z, dt_bias=w["b_dt"], init=ssm0, chunk_states=train, **k)
    o, _ = rsm.linear(y, w["w_out"])
    return o, s, (conv1, ssm1), dict(u=u, xz=xz, c=c, p=p, dt=dt, y=y, states=states, conv0=conv0, ssm0=ssm0)


def oracle_block(w, stream, x, lens, R, N, dtype, init=None):
    """The same in 64 bits, on the weights' stored values; the stream is what the sum is rounded to."""
    import torch
    W = {k: f64(t) for k, t in w.items()}
    inner = W["conv_w"].shape[0]
    s = f64((x.double() + stream.double()).to(x.dtype))
    u = O.rms_norm(s, W["norm"])
    xz = u @ W["w_in"].T
    out = dict(o=np.zeros_like(s), s=s, final=[])
    at = 0
    for i, n in enumerate(lens):
        zero = np.zeros((3, inner)) if init is None else f64(init[0])[i]
        a = xz[at:at + n, :inner]
        c, f, _ = O.conv(a, W["conv_w"], W["conv_b"], zero, "silu")
        p = c @ W["w_x"].T
        dt = p[:, :R] @ W["w_dt"].T
        r = O.ssm(c, dt, W["A"], p[:, R:R + N], p[:, R + N:], W["D"], xz[at:at + n, inner:], W["b_dt"],
                  init=None if init is None else f64(init[1])[i])
        out["o"][at:at + n] = r["y"] @ W["w_out"].T
        out["final"].append((f, r["final"]))
        at += n
    return out


@pytest.mark.parametrize("dtype,bits", [("bf16", False), ("fp32", False), ("bf16", True)])
def test_prompt_and_single_tokens(dtype, bits):
    """Packed prompts, then tokens one at a time from the states they leave."""
    import torch
    import recurrent_sequence_models_amd as rsm
    d, inner, N, R, lens, more = 128, 256, 16, 16, [70, 0, 3, 130], 3
    w = weights(d, inner, N, R, dtype)
    n, total = len(lens), sum(lens)
    stream, x = rand(50, total, d, dtype=dtype), rand(51, total, d, dtype=dtype)
    o, s, state, _ = block(rsm, w, stream, x, offsets(lens), R, N, bits=bits)
    ref = oracle_block(w, stream, x, lens, R, N, dtype)
    # e4m3 keeps 4 bits: operands are off by up to 2^-4, 2^-4 / sqrt(3) in the mean, each
    bar = 0.06 if bits else TOL[dtype]
    assert rel_l2(f64(o), ref["o"]) <= bar and rel_l2(f64(s), ref["s"]) <= 1e-12
    for i in range(n):
        for got, want in zip((state[0][i], state[1][i]), ref["final"][i]):
            assert np.linalg.norm(f64(got) - want) <= bar * np.linalg.norm(want) + 1e-30
    inner_of = w["conv_w"].shape[0]
    conv, ssm = state
    for t in range(more):
        st, xt = rand(60 + t, n, d, dtype=dtype), rand(70 + t, n, d, dtype=dtype)
        want = oracle_block(w, st, xt, [1] * n, R, N, dtype, init=(conv, ssm))
        if bits:
            u, s1, scale = rsm.rms_norm(xt, w["norm"], residual=st, quantize=True)
            q, qs = rsm.quantize_rows(w["w_in"])
            xz, _ = rsm.linear(u, q, x_scale=scale, weight_scale=qs, out_dtype=xt.dtype)
        else:
            u, s1, _ = rsm.rms_norm(xt, w["norm"], residual=st)
            xz, _ = rsm.linear(u, w["w_in"])
        c = rsm.causal_conv_step(xz[:, :inner_of], w["conv_w"], conv, bias=w["conv_b"], activation="silu")
        p, _ = rsm.linear(c, w["w_x"])
        dt, _ = rsm.linear(p[:, :R], w["w_dt"])
        y = rsm.selective_scan_step(c, dt, w["A"], p[:, R:R + N], p[:, R + N:], ssm, D=w["D"], z=xz[:, inner_of:], dt_bias=w["b_dt"])
        out, _ = rsm.linear(y, w["w_out"], residual=s1)
        assert rel_l2(f64(out), want["o"] + want["s"]) <= bar
        for i in range(n):
            for got, to in zip((conv[i], ssm[i]), want["final"][i]):
                assert np.linalg.norm(f64(got) - to) <= bar * np.linalg.norm(to) + 1e-30


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_training(dtype):
    """All gradients of a block, against torch's automatic differentiation of the same formulas in 64 bits."""
    import torch
    import recurrent_sequence_models_amd as rsm
    d, inner, N, R, lens = 64, 128, 16, 16, [40, 1, 100]
    total = sum(lens)
    w = weights(d, inner, N, R, dtype, seed=20)
    stream, x, do, ds = (rand(i, total, d, dtype=dtype) for i in (80, 81, 82, 83))
    cu = offsets(lens)
    o, s, _, k = block(rsm, w, stream, x, cu, R, N, train=True)
    # back through the block; gradients of views of a projection are written into one array
    g = {}
    a = rsm.linear_bwd(k["y"], w["w_out"], do)
    g["w_out"] = a["dweight"]
    dxz, dp = torch.empty_like(k["xz"]), torch.empty_like(k["p"])
    xs, z = k["xz"][:, :inner], k["xz"][:, inner:]
    B, C = k["p"][:, R:R + N], k["p"][:, R + N:]
    dc, ddt = torch.empty_like(k["c"]), torch.empty_like(k["dt"])
    b = rsm.selective_scan_bwd(k["c"], k["dt"], w["A"], B, C, a["dx"], k["states"], D=w["D"], z=z, dt_bias=w["b_dt"], cu_seqlens=cu,
                               out=dict(dx=dc, ddt=ddt, dB=dp[:, R:R + N], dC=dp[:, R + N:], dz=dxz[:, inner:]))
    g.update(A=b["dA"], D=b["dD"], b_dt=b["ddt_bias"])
    a = rsm.linear_bwd(k["p"][:, :R], w["w_dt"], ddt, dx=dp[:, :R])
    g["w_dt"] = a["dweight"]
    a = rsm.linear_bwd(k["c"], w["w_x"], dp)
    g["w_x"] = a["dweight"]
    dc += a["dx"]
    b = rsm.causal_conv_bwd(xs, w["conv_w"], dc, bias=w["conv_b"], activation="silu", cu_seqlens=cu, out=dxz[:, :inner])
    g.update(conv_w=b["dweight"], conv_b=b["dbias"])
    a = rsm.linear_bwd(k["u"], w["w_in"], dxz)
    g["w_in"] = a["dweight"]
    b = rsm.rms_norm_bwd(s, w["norm"], a["dx"], d_stream=ds)
    g.update(norm=b["dweight"], x=b["dx"])
    torch.cuda.synchronize()

    p = {n: t.double().cpu().requires_grad_() for n, t in w.items()}
    sv = s.double().cpu().requires_grad_()
    u = sv * p["norm"] * torch.rsqrt((sv * sv).mean(-1, keepdim=True) + 1e-6)
    xz = u @ p["w_in"].T
    outs, at = [], 0
    for n in lens:
        ext = torch.cat([torch.zeros(3, inner, dtype=torch.float64), xz[at:at + n, :inner]])
        c = sum(p["conv_w"][:, j] * ext[j:j + n] for j in range(4)) + p["conv_b"]
        c = c * torch.sigmoid(c)
        q = c @ p["w_x"].T
        delta = torch.nn.functional.softplus(q[:, :R] @ p["w_dt"].T + p["b_dt"], threshold=1000)
        h = torch.zeros(inner, N, dtype=torch.float64)
        ys = []
        for t in range(n):
            h = torch.exp(delta[t][:, None] * p["A"]) * h + (delta[t] * c[t])[:, None] * q[t, R:R + N]
            ys.append((h * q[t, R + N:]).sum(-1) + p["D"] * c[t])
        zz = xz[at:at + n, inner:]
        outs.append(torch.stack(ys) * zz * torch.sigmoid(zz))
        at += n
    want_o = torch.cat(outs) @ p["w_out"].T
    loss = (do.double().cpu() * want_o).sum() + (ds.double().cpu() * sv).sum()
    names = list(p)
    grads = torch.autograd.grad(loss, [sv] + [p[n] for n in names])
    assert rel_l2(f64(o), want_o.detach().numpy()) <= TOL[dtype]
    for name, want in zip(["x"] + names, grads):
        assert rel_l2(f64(g[name]), want.numpy()) <= TOL[dtype], name


def test_graphs_that_share_a_workspace():
    """Two captured graphs whose calls were given the same workspaces, replayed in turn with eager calls on
    them between."""
    import torch
    import recurrent_sequence_models_amd as rsm
    B, T, D, N = 1, 900, 64, 16
    x, dt, z, dy = (rand(i, B, T, D, dtype="bf16") for i in range(4))
    Bm, Cm = rand(5, B, T, N, dtype="bf16"), rand(6, B, T, N, dtype="bf16")
    A, bias, w4 = -torch.exp(rand(7, D, N)), rand(8, D), rand(9, D, 4)
    W, v, nw = rand(10, 128, 2048, dtype="bf16"), rand(11, 200, 2048, dtype="bf16"), rand(12, D)
    ws = [torch.empty(1 << 25, dtype=torch.uint8, device="cuda") for _ in range(5)]

    def call(second):
        act = "silu" if second else "gelu"
        y, fin, st = rsm.selective_scan(x, dt, A, Bm, Cm, z=z, dt_bias=bias if second else None, chunk_states=True, workspace=ws[0])
        g = rsm.selective_scan_bwd(x, dt, A, Bm, Cm, dy, st, z=z, dt_bias=bias if second else None, workspace=ws[1])
        c = rsm.causal_conv_bwd(x, w4, dy, activation="silu" if second else None, workspace=ws[2])
        o, pre = rsm.linear(v, W, activation=act, pre=True, workspace=ws[3])
        l = rsm.linear_bwd(v, W, o, pre=pre, activation=act, bias=second, workspace=ws[3])
        n = rsm.rms_norm_bwd(x, nw, dy, d_stream=z if second else None, workspace=ws[4])
        return [t for t in [y, fin, *g.values(), *c.values(), o, pre, *l.values(), *n.values()] if t is not None]

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
        for a, b in zip(got[turn], want[turn]):
            assert torch.equal(a, b)
        for a, b in zip(eager, want[not turn]):
            assert torch.equal(a, b)
