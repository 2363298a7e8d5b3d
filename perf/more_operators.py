"""Workloads of the operators of a state-space block: the norm of the residual stream (with an output
in 8 bits for the products behind it), the projections with their epilogues, the short causal
convolution and the selective state-space scan.

``listed()`` names the workloads, ``draw`` makes more of the same ranges, ``prepare`` makes the
inputs, ``run`` is one pass: through the library's entry points where ``own`` is true, else in
elementary torch operations.  ``exact`` is the same pass from the definitions in 64 bits.

Sizes: width 768 at 8 x 2048 and 4 x 4096 tokens are the 130M layer of the benchmark, width 2048 its
long-context workload; a block's inner width is twice the model's, with 16 states a channel.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------

def _norm(kind, dtype, tokens, width, residual=True):
    return dict(op="norm", kind=kind, dtype=dtype, tokens=tokens, width=width, residual=residual)


def _conv(kind, dtype, B, T, D, taps=4, silu=True, packed=0):
    return dict(op="conv", kind=kind, dtype=dtype, B=B, T=T, D=D, taps=taps, silu=silu, packed=packed)


def _scan(kind, dtype, B, T, D, N=16, gate=True, packed=0):
    return dict(op="scan", kind=kind, dtype=dtype, B=B, T=T, D=D, N=N, gate=gate, packed=packed)


def _linear(kind, dtype, tokens, K, N, act="none", bias=True, residual=False):
    return dict(op="linear", kind=kind, dtype=dtype, tokens=tokens, K=K, N=N, act=act, bias=bias, residual=residual)


def listed():
    return [
        # one token for each of 64 sequences of a decoding server: the stream's norm, in 8 bits for the projection
        dict(_norm("q8", "bf16", 64, 2048), name="norm_token"),
        # the norm before a layer in a training step, with the stream's own gradient coming in
        dict(_norm("train", "bf16", 16387, 2048), name="norm_train"),
        # the decoding server's inner activations through the convolution
        dict(_conv("step", "bf16", 64, 1, 4096), name="conv_token"),
        # a training step of the 130M block's convolution
        dict(_conv("train", "bf16", 4, 4096, 1536), name="conv_train"),
        # the decoding server's states, one token each
        dict(_scan("step", "bf16", 64, 1, 4096), name="scan_token"),
        # the 130M block's scan over its benchmark batch
        dict(_scan("fwd", "bf16", 8, 2048, 1536), name="scan_layer"),
        # a server's prompts of different lengths, packed, in full precision
        dict(_scan("fwd", "fp32", 1, 5003, 4096, packed=13), name="scan_packed"),
        # a training step of the 130M block's scan
        dict(_scan("train", "bf16", 4, 4096, 1536), name="scan_train"),
        # a few decoding sequences through a projection
        dict(_linear("fwd", "bf16", 16, 2048, 4096, residual=False), name="linear_token"),
        # the projection into a block of width 2048, with its activation
        dict(_linear("fwd", "bf16", 16384, 2048, 4096, act="silu"), name="linear_layer"),
        # the projection back to the stream on 8-bit activations and weights, added to the residual
        dict(_linear("q8", "bf16", 16387, 4096, 2048, residual=True), name="linear_8bit"),
        # a training step of the 130M block's projection
        dict(_linear("train", "bf16", 16384, 768, 1536, act="silu"), name="linear_train"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "conv", "scan", "scan", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "norm":
        width = 8 * _log_int(rng, 8, 1024)
        return _norm(rng.choice(["fwd", "q8", "train"]), dtype, _log_int(rng, 1, min(32768, (32 << 20) // width)), width,
                     residual=rng.random() < 0.7)
    if op == "linear":
        kind = rng.choice(["fwd", "fwd", "q8", "train"])
        tokens, K, N = _log_int(rng, 1, 16384), 16 * _log_int(rng, 4, 256), 8 * _log_int(rng, 8, 512)
        if dtype == "fp32" and kind != "q8":          # at most 2^35 products of two numbers
            tokens = min(tokens, max(1, (1 << 35) // (K * N)))
        return _linear(kind, dtype, tokens, K, N, act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.7,
                       residual=rng.random() < 0.5 and kind != "train")
    kind = rng.choice(["step", "fwd", "fwd", "train"])
    D = 8 * _log_int(rng, 8, 512)
    N = rng.choice([16, 16, 16, 32, 64]) if op == "scan" else 1
    if kind == "step":
        B = _log_int(rng, 1, 256)
        if op == "conv":
            return _conv(kind, dtype, B, 1, D, taps=rng.randint(2, 4), silu=rng.random() < 0.7)
        return _scan(kind, dtype, B, 1, D, N=N, gate=rng.random() < 0.7)
    most = (1 << 28) // (D * N) if op == "scan" else (1 << 25) // D      # tokens
    T = _log_int(rng, 1, min(16384, most))
    B, packed = rng.randint(1, max(1, min(32, most // T))), 0
    if rng.random() < 0.4:
        T, B = min(T * B, 16384), 1
        packed = rng.randint(1, min(T, 40))
    if op == "conv":
        return _conv(kind, dtype, B, T, D, taps=rng.randint(2, 4), silu=rng.random() < 0.7, packed=packed)
    return _scan(kind, dtype, B, T, D, N=N, gate=rng.random() < 0.7, packed=packed)


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------

def _lens(case):
    """The sequences' lengths, the same for every seed."""
    if not case["packed"]:
        return [case["T"]] * case["B"]
    total, n = case["T"], case["packed"]
    r = random.Random(total * 1009 + n)
    at = sorted(r.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + at, at + [total])]


def _offsets(lens, dev):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62))
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    s = dict(case=case)
    kind = case["kind"]
    if case["op"] == "norm":
        shape = (case["tokens"], case["width"])
        s["x"], s["w"] = normal(*shape, dtype=dt), 1 + 0.2 * normal(case["width"])
        s["res"] = normal(*shape, dtype=dt, scale=3.0) if case["residual"] else None
        if kind == "train":
            s["dy"], s["ds"] = normal(*shape, dtype=dt), normal(*shape, dtype=dt)
        return s
    if case["op"] == "linear":
        M, K, N = case["tokens"], case["K"], case["N"]
        s["bias"] = normal(N, scale=0.5) if case["bias"] else None
        s["res"] = normal(M, N, dtype=dt) if case["residual"] else None
        x, w = normal(M, K), normal(N, K, scale=K ** -0.5)
        if kind == "q8":    # quantised by the rows' largest entries, as the norm leaves activations
            for name, t in (("x", x), ("w", w)):
                scale = t.abs().amax(-1) / F8_MAX
                s[name], s[name + "_scale"] = (t / scale[:, None]).to(F8), scale
        else:
            s["x"], s["w"] = x.to(dt), w.to(dt)
        if kind == "train":
            s["dy"] = normal(M, N, dtype=dt)
        return s
    lens, D = _lens(case), case["D"]
    n = len(lens)
    lead = (n,) if kind == "step" else (case["T"],) if case["packed"] else (n, case["T"])
    if kind != "step":
        s["lens"] = lens
        s["cu"] = _offsets(lens, dev) if case["packed"] else None
    s["x"] = normal(*lead, D, dtype=dt)
    if case["op"] == "conv":
        W = case["taps"]
        s["w"], s["bias"] = normal(D, W, scale=W ** -0.5), normal(D, scale=0.2)
        s["init"] = normal(n, W - 1, D, dtype=dt)
        if kind == "train":
            s["dy"], s["dfinal"] = normal(*lead, D, dtype=dt), normal(n, W - 1, D, dtype=dt)
        return s
    # steps between 0.001 and 0.1 at a zero dt, decays -1 .. -N as such layers start from
    N = case["N"]
    step = torch.exp(torch.rand(D, generator=g, device=dev) * math.log(100.0) + math.log(0.001))
    s["bias"] = torch.log(torch.expm1(step))
    s["dt"] = normal(*lead, D, dtype=dt, scale=0.5)
    s["A"] = -torch.arange(1, N + 1, device=dev) * torch.exp(normal(D, N, scale=0.1))
    s["B"], s["C"] = normal(*lead, N, dtype=dt), normal(*lead, N, dtype=dt)
    s["D"] = 1 + 0.2 * normal(D)
    s["z"] = normal(*lead, D, dtype=dt) if case["gate"] else None
    s["init"] = normal(n, D, N, scale=0.3)
    if kind == "train":
        s["dy"], s["dfinal"] = normal(*lead, D, dtype=dt), normal(n, D, N, scale=0.3)
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if case["op"] == "norm":
        n, w = case["tokens"] * case["width"], 4 * case["width"]
        r = 2 if case["residual"] else 0               # the residual in, the stream out
        if kind == "train":                            # x, dy, ds in; y, dx out
            return dict(bytes=(5 + r) * n * e + 2 * w, flops=14 * n)
        out = n + 4 * case["tokens"] if kind == "q8" else n * e
        return dict(bytes=(1 + r) * n * e + out + w, flops=5 * n)
    if case["op"] == "linear":
        M, K, N = case["tokens"], case["K"], case["N"]
        a = 1 if kind == "q8" else e
        size = a * (M * K + N * K) + e * M * N * (2 if case["residual"] else 1) + 4 * (N if case["bias"] else 0)
        if kind == "train":                            # dy in; dx, dw, db out
            return dict(bytes=size + e * (M * N + M * K + N * K) + 4 * N, flops=6 * M * K * N)
        return dict(bytes=size, flops=2 * M * K * N)
    tokens = case["B"] * case["T"]
    seqs, D = case["packed"] or case["B"], case["D"]
    n = tokens * D
    if case["op"] == "conv":
        W = case["taps"]
        state, par = seqs * (W - 1) * D * e, 4 * D * (W + 1)
        if kind == "train":                            # x, dy in; y, dx out
            return dict(bytes=4 * n * e + 4 * state + 2 * par, flops=n * (6 * W + 16))
        return dict(bytes=2 * n * e + 2 * state + par, flops=n * (2 * W + 5))
    N = case["N"]
    z = 1 if case["gate"] else 0
    state, par = 4 * seqs * D * N, 4 * D * (N + 2)
    fwd = (3 + z) * n * e + 2 * tokens * N * e + 2 * state + par       # x, dt, z in, y out; B, C
    if kind == "train":                                # dy in; dx, ddt, dz, dB, dC out
        return dict(bytes=fwd + (3 + z) * n * e + 2 * tokens * N * e + 2 * state + par, flops=26 * n * N)
    return dict(bytes=fwd, flops=7 * n * N)


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------

def run(s):
    return dict(norm=_run_norm, linear=_run_linear, conv=_run_conv, scan=_run_scan)[s["case"]["op"]](s)


def _run_norm(s):
    c = s["case"]
    if own:
        import recurrent_sequence_models_amd as rsm
        y, stream, scale = rsm.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, quantize=c["kind"] == "q8")
        out = dict(y=y, stream=stream if c["residual"] else None, scale=scale)
        if c["kind"] == "train":
            g = rsm.rms_norm_bwd(stream, s["w"], s["dy"], d_stream=s["ds"], eps=EPS)
            out.update(dx=g["dx"], dw=g["dweight"])
        return out
    dt = s["x"].dtype
    # the stream is what the sum is rounded to, and the norm is of the stream
    stream = (s["x"].float() + s["res"].float()).to(dt) if c["residual"] else s["x"]
    v = stream.float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    y = v * r * s["w"]
    out = dict(y=y.to(dt), stream=stream if c["residual"] else None, scale=None)
    if c["kind"] == "q8":
        out["scale"] = y.abs().amax(-1).clamp(min=1e-30) / F8_MAX
        out["y"] = (y / out["scale"][:, None]).to(F8)
    if c["kind"] == "train":
        dy, vr = s["dy"].float(), v * r
        wu = s["w"] * dy
        dx = r * (wu - vr * (wu * vr).mean(-1, keepdim=True)) + s["ds"].float()
        out.update(dx=dx.to(dt), dw=(dy * vr).sum(0, dtype=torch.float64).float())
    return out


def _act(v, act):
    """(the activation, its derivative)."""
    if act == "silu":
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(v * 0.5 ** 0.5))
        return v * p, p + v * torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5
    return v, torch.ones_like(v)


def _run_linear(s):
    c = s["case"]
    act = None if c["act"] == "none" else c["act"]
    train = c["kind"] == "train"
    if own:
        import recurrent_sequence_models_amd as rsm
        scales = dict(x_scale=s["x_scale"], weight_scale=s["w_scale"], out_dtype=DT[c["dtype"]]) if c["kind"] == "q8" else {}
        y, pre = rsm.linear(s["x"], s["w"], bias=s["bias"], activation=act, residual=s["res"], pre=train and act is not None,
                            **scales)
        if not train:
            return dict(y=y)
        g = rsm.linear_bwd(s["x"], s["w"], s["dy"], pre=pre, activation=act, bias=c["bias"])
        return dict(y=y, dx=g["dx"], dw=g["dweight"], db=g["dbias"])
    dt = DT[c["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    v = x @ w.T
    if c["kind"] == "q8":
        v = v * s["x_scale"][:, None] * s["w_scale"]
    if c["bias"]:
        v = v + s["bias"]
    y, slope = _act(v, c["act"])
    if c["residual"]:
        y = y + s["res"].float()
    if not train:
        return dict(y=y.to(dt))
    d = s["dy"].float() * slope
    return dict(y=y.to(dt), dx=(d @ w).to(dt), dw=(d.T @ x).to(dt), db=d.sum(0, dtype=torch.float64).float() if c["bias"] else None)


def _run_conv(s):
    c = s["case"]
    W, D, dt = c["taps"], c["D"], s["x"].dtype
    act = "silu" if c["silu"] else None
    if own:
        import recurrent_sequence_models_amd as rsm
        if c["kind"] == "step":
            state = torch.empty_like(s["init"])
            return dict(y=rsm.causal_conv_step(s["x"], s["w"], s["init"], bias=s["bias"], activation=act, state_out=state),
                        final=state)
        y, final = rsm.causal_conv(s["x"], s["w"], bias=s["bias"], activation=act, cu_seqlens=s["cu"], init=s["init"])
        if c["kind"] != "train":
            return dict(y=y, final=final)
        g = rsm.causal_conv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], activation=act, cu_seqlens=s["cu"], init=s["init"],
                                d_final=s["dfinal"])
        return dict(y=y, final=final, dx=g["dx"], dw=g["dweight"], db=g["dbias"], dinit=g["d_init"])
    w = s["w"].T                                        # [W, D]
    if c["kind"] == "step":
        win = torch.cat([s["init"], s["x"][:, None]], 1)
        v = (win.float() * w).sum(1) + s["bias"]
        return dict(y=_act(v, "silu" if c["silu"] else "none")[0].to(dt), final=win[:, 1:].contiguous())
    # the sequences on one time axis, each behind the W - 1 inputs that it starts from
    dev, lens = s["x"].device, torch.tensor(s["lens"], device=s["x"].device)
    n = len(s["lens"])
    seq = torch.repeat_interleave(torch.arange(n, device=dev), lens)
    at = torch.arange(seq.numel(), device=dev) + (seq + 1) * (W - 1)
    ends = torch.cumsum(lens, 0) + torch.arange(1, n + 1, device=dev) * (W - 1)
    taps = torch.arange(W, device=dev)
    first = (ends - lens - (W - 1))[:, None] + taps[:-1]
    last = ends[:, None] - (W - 1) + taps[:-1]
    ext = torch.zeros(seq.numel() + n * (W - 1), D, device=dev)
    ext[at], ext[first] = s["x"].reshape(-1, D).float(), s["init"].float()
    win = ext[at[:, None] - (W - 1) + taps]
    y, slope = _act((win * w).sum(1) + s["bias"], "silu" if c["silu"] else "none")
    out = dict(y=y.to(dt).view_as(s["x"]), final=ext[last].to(dt))
    if c["kind"] == "train":
        d = s["dy"].reshape(-1, D).float() * slope
        dext = torch.zeros(ext.shape[0] + W - 1, D, device=dev)
        dext[at] = d
        back = (dext[torch.arange(ext.shape[0], device=dev)[:, None] + taps] * w.flip(0)).sum(1)
        back[last] += s["dfinal"].float()
        out.update(dx=back[at].to(dt).view_as(s["x"]), dinit=back[first].to(dt), db=d.sum(0, dtype=torch.float64).float(),
                   dw=(d[:, None] * win).sum(0, dtype=torch.float64).float().T.contiguous())
    return out


def _doubling(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 0 from h = 0, by doubling spans."""
    k = 1
    while k < u.shape[0]:
        u = torch.cat([u[:k], u[k:] + a[k:] * u[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return u


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _run_scan(s):
    c = s["case"]
    if own:
        import recurrent_sequence_models_amd as rsm
        kw = dict(D=s["D"], z=s["z"], dt_bias=s["bias"], softplus=True)
        args = s["x"], s["dt"], s["A"], s["B"], s["C"]
        if c["kind"] == "step":
            state = torch.empty_like(s["init"])
            return dict(y=rsm.selective_scan_step(*args, s["init"], state_out=state, **kw), final=state)
        kw.update(cu_seqlens=s["cu"], init=s["init"])
        train = c["kind"] == "train"
        y, final, states = rsm.selective_scan(*args, chunk_states=train, **kw)
        if not train:
            return dict(y=y, final=final)
        g = rsm.selective_scan_bwd(*args, s["dy"], states, d_final=s["dfinal"], **kw)
        return dict(y=y, final=final, dx=g["dx"], ddt=g["ddt"], dA=g["dA"], dB=g["dB"], dC=g["dC"], dD=g["dD"], dz=g["dz"],
                    dbias=g["ddt_bias"], dinit=g["d_init"])
    dt, D, N = s["x"].dtype, c["D"], c["N"]
    # the sequences on one time axis
    x, B, C = s["x"].reshape(-1, D).float(), s["B"].reshape(-1, N).float(), s["C"].reshape(-1, N).float()
    raw = s["dt"].reshape(-1, D).float() + s["bias"]
    delta = _softplus(raw)
    a = torch.exp(delta[..., None] * s["A"])
    u = (delta * x)[..., None] * B[:, None]
    dev = x.device
    lens = torch.tensor(s["lens"] if c["kind"] != "step" else [1] * x.shape[0], device=dev)
    last = torch.cumsum(lens, 0) - 1
    first = last - lens + 1
    u[first] += a[first] * s["init"]
    begin = a[first]
    cut = a.clone()
    cut[first] = 0
    h = _doubling(cut, u)
    read = (h * C[:, None]).sum(-1) + s["D"] * x
    gate, slope = _act(s["z"].reshape(-1, D).float(), "silu") if c["gate"] else (1.0, None)
    out = dict(y=(read * gate).to(dt).view_as(s["x"]), final=h[last])
    if c["kind"] != "train":
        return out
    dy = s["dy"].reshape(-1, D).float()
    gy = dy * gate
    w = gy[..., None] * C[:, None]
    w[last] += s["dfinal"]
    nxt = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    g = torch.flip(_doubling(torch.flip(nxt, [0]), torch.flip(w, [0])), [0])
    del w, nxt, u, cut
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[first] = s["init"]
    ah = g * a * prev
    gb = (g * B[:, None]).sum(-1)
    ddt = ((ah * s["A"]).sum(-1) + gb * x) * torch.sigmoid(raw)
    out.update(dx=(gb * delta + s["D"] * gy).to(dt).view_as(s["x"]), ddt=ddt.to(dt).view_as(s["x"]),
               dA=(ah * delta[..., None]).sum(0, dtype=torch.float64).float(),
               dB=(g * (delta * x)[..., None]).sum(1).to(dt).view_as(s["B"]), dC=(h * gy[..., None]).sum(1).to(dt).view_as(s["C"]),
               dD=(gy * x).sum(0, dtype=torch.float64).float(), dbias=ddt.sum(0, dtype=torch.float64).float(),
               dz=(dy * read * slope).to(dt).view_as(s["x"]) if c["gate"] else None, dinit=begin * g[first])
    return out


# ---------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, linear=_exact_linear, conv=_exact_conv, scan=_exact_scan)[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    w = s["w"].double()
    v = s["x"].double()
    out = dict(y=None, stream=None, scale=None)
    if c["residual"]:      # the stream is held in the inputs' type
        v = v + s["res"].double()
        out["stream"] = v
        v = v.to(s["x"].dtype).double()
    ms = v.square().sum(-1, keepdim=True) / c["width"] + EPS
    out["y"] = w * v / ms.sqrt()
    if c["kind"] == "q8":  # in units of the row's scale, before the rounding to 8 bits
        out["scale"] = out["y"].abs().amax(-1) / F8_MAX
        out["y"] = out["y"] / out["scale"][:, None]
    if c["kind"] == "train":
        dy = s["dy"].double()
        inner = (dy * w * v).sum(-1, keepdim=True) / c["width"]
        out.update(dx=dy * w / ms.sqrt() - v * inner / ms ** 1.5 + s["ds"].double(), dw=(dy * v / ms.sqrt()).sum(0))
    return out


def _exact_act(v, act):
    v = v.detach().requires_grad_()
    y = torch.nn.functional.silu(v) if act == "silu" else torch.nn.functional.gelu(v) if act == "gelu" else v * 1.0
    slope, = torch.autograd.grad(y.sum(), v)
    return y.detach(), slope


def _exact_linear(s):
    c = s["case"]
    x, w = s["x"].double(), s["w"].double()
    if c["kind"] == "q8":
        x, w = x * s["x_scale"].double()[:, None], w * s["w_scale"].double()[:, None]
    v = x @ w.T + (s["bias"].double() if c["bias"] else 0)
    y, slope = _exact_act(v, c["act"])
    if c["residual"]:
        y = y + s["res"].double()
    if c["kind"] != "train":
        return dict(y=y)
    d = s["dy"].double() * slope
    return dict(y=y, dx=d @ w, dw=d.T @ x, db=d.sum(0) if c["bias"] else None)


def _exact_conv(s):
    c = s["case"]
    W, D = c["taps"], c["D"]
    w, b, act = s["w"].double(), s["bias"].double(), "silu" if c["silu"] else "none"
    step = c["kind"] == "step"
    x, init = s["x"].double().reshape(-1, D), s["init"].double()
    lens = [1] * x.shape[0] if step else s["lens"]
    keep = {k: [] for k in ("y", "final", "dx", "dinit")}
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    at = 0
    for i, n in enumerate(lens):
        ext = torch.cat([init[i], x[at:at + n]])
        win = ext.unfold(0, W, 1)                        # [n, D, W]
        y, slope = _exact_act((win * w).sum(-1) + b, act)
        keep["y"].append(y)
        keep["final"].append(ext[n:])
        if c["kind"] == "train":
            d = s["dy"].reshape(-1, D)[at:at + n].double() * slope
            dw += (d[..., None] * win).sum(0)
            db += d.sum(0)
            back = torch.zeros_like(ext)
            for j in range(W):
                back[j:j + n] += d * w[:, j]
            back[n:] += s["dfinal"][i].double()
            keep["dx"].append(back[W - 1:])
            keep["dinit"].append(back[:W - 1])
        at += n
    out = dict(y=torch.cat(keep["y"]).view(s["x"].shape), final=torch.stack(keep["final"]))
    if c["kind"] == "train":
        out.update(dx=torch.cat(keep["dx"]).view(s["x"].shape), dinit=torch.stack(keep["dinit"]), dw=dw, db=db)
    return out


def _exact_scan(s):
    c = s["case"]
    D, N = c["D"], c["N"]
    step, train = c["kind"] == "step", c["kind"] == "train"
    # sequences side by side, [longest, n, ...], each from its own first step (backward: the same places)
    lens = [1] * s["x"].shape[0] if step else s["lens"]
    n, T = len(lens), max(lens)
    dev = s["x"].device
    ls = torch.tensor(lens, device=dev)
    start = torch.cumsum(ls, 0) - ls
    here = torch.arange(T, device=dev)[:, None] < ls
    idx = (start + torch.arange(T, device=dev)[:, None]).clamp(max=int(ls.sum()) - 1)

    def side(t, width):
        return t.reshape(-1, width)[idx].double()

    x, B, C = side(s["x"], D), side(s["B"], N), side(s["C"], N)
    raw = side(s["dt"], D) + s["bias"].double()
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    A, skip = s["A"].double(), s["D"].double()
    h = s["init"].double()
    hs = torch.empty(T + 1 if train else 1, n, D, N, dtype=torch.float64, device=dev)
    hs[0] = h
    read = torch.empty(T, n, D, dtype=torch.float64, device=dev)
    for t in range(T):
        new = torch.exp(delta[t][..., None] * A) * h + (delta[t] * x[t])[..., None] * B[t][:, None]
        h = torch.where(here[t][:, None, None], new, h)
        read[t] = torch.einsum("ndk,nk->nd", h, C[t]) + skip * x[t]
        if train:
            hs[t + 1] = h
    z = side(s["z"], D) if c["gate"] else None
    gate, slope = _exact_act(z, "silu") if c["gate"] else (1.0, None)

    def flat(t):
        return t.transpose(0, 1)[here.T].reshape(s["x"].shape[:-1] + t.shape[-1:])

    out = dict(y=flat(read * gate), final=h)
    if not train:
        return out
    dy = side(s["dy"], D) * here[..., None]
    gy = dy * gate
    dx, ddt, dB, dC = (torch.zeros_like(t) for t in (x, x, B, C))
    dA = torch.zeros_like(A)
    g = s["dfinal"].double()
    for t in range(T - 1, -1, -1):
        on = here[t][:, None, None]
        gt = g + gy[t][..., None] * C[t][:, None]
        r = torch.exp(delta[t][..., None] * A) * gt
        gt = torch.where(on, gt, torch.zeros_like(gt))
        ah = torch.where(on, r * hs[t], torch.zeros_like(gt))
        gb = torch.einsum("ndk,nk->nd", gt, B[t])
        dx[t] = gb * delta[t] + skip * gy[t]
        ddt[t] = ((ah * A).sum(-1) + gb * x[t]) * torch.sigmoid(raw[t])
        dA += (ah * delta[t][..., None]).sum(0)
        dB[t] = torch.einsum("ndk,nd->nk", gt, delta[t] * x[t])
        dC[t] = torch.einsum("ndk,nd->nk", hs[t + 1], gy[t])
        g = torch.where(on, r, g)
    out.update(dx=flat(dx), ddt=flat(ddt), dA=dA, dB=flat(dB), dC=flat(dC), dD=(gy * x).sum((0, 1)), dbias=ddt.sum((0, 1)),
               dz=flat(dy * read * slope) if c["gate"] else None, dinit=g)
    return out
