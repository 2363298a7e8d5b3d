"""Workloads of the layer operators: the gated linear recurrence, the query / key head norm with
rotary positions, and causal attention over packed sequences.

``listed()`` names the workloads, ``draw`` makes more of the same ranges, ``prepare`` makes the
inputs, ``run`` is one pass: through the library's entry points where ``own`` is true, else in
elementary torch operations.  ``exact`` is the same pass from the definitions in 64 bits.

Sizes: 12 heads of 64 at width 768 are the 130M layer of the benchmark; 16 heads of 128 (width 2048)
and 65 536 tokens its long-context workload.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------

def _scan(kind, dtype, B, T, D, packed=0, mix=False):
    return dict(op="scan", kind=kind, dtype=dtype, B=B, T=T, D=D, packed=packed, mix=mix)


def _qk(kind, dtype, tokens, hq, hk, d, rot, layout, far, up="same"):
    return dict(op="qk", kind=kind, dtype=dtype, tokens=tokens, hq=hq, hk=hk, d=d, rot=rot, layout=layout, far=far,
                up=up)


def _attn(kind, dtype, n, lq, hq, hk, d, ragged=False, prefix=0):
    return dict(op="attn", kind=kind, dtype=dtype, n=n, lq=lq, hq=hq, hk=hk, d=d, ragged=ragged, prefix=prefix)


def listed():
    return [
        # one token for each of 64 sequences of a decoding server, width 2048
        dict(_scan("step", "bf16", 64, 1, 2048), name="scan_step"),
        # a recurrence layer of the 130M model over its benchmark batch
        dict(_scan("fwd", "bf16", 8, 2048, 768, mix=True), name="scan_layer"),
        # a server's prompts of different lengths, packed, in full precision
        dict(_scan("fwd", "fp32", 1, 9001, 2048, packed=13), name="scan_packed"),
        # one long document
        dict(_scan("fwd", "bf16", 1, 65536, 2048), name="scan_long"),
        # a training step of the layer: forward and backward
        dict(_scan("train", "bf16", 4, 4096, 768, mix=True), name="scan_train"),
        # the decoding server's queries and keys at far positions
        dict(_qk("fwd", "bf16", 64, 16, 4, 128, 128, "half", 65536), name="qk_token"),
        # queries and keys of the 130M layer's batch
        dict(_qk("fwd", "bf16", 16384, 12, 12, 64, 64, "half", 2048), name="qk_layer"),
        # the backward of grouped heads, half of each head rotated, single-precision gradients coming in
        dict(_qk("bwd", "bf16", 16387, 16, 4, 128, 64, "interleaved", 65536, up="fp32"), name="qk_bwd"),
        # a few short prompts of a small model
        dict(_attn("fwd", "bf16", 7, 211, 12, 12, 64, ragged=True), name="attn_ragged"),
        # one long prompt with grouped heads
        dict(_attn("fwd", "bf16", 1, 16384, 16, 4, 128), name="attn_long"),
        # single tokens against long contexts
        dict(_attn("fwd", "bf16", 16, 1, 16, 4, 128, ragged=True, prefix=16384), name="attn_token"),
        # a training step of an attention layer at the benchmark's batch
        dict(_attn("train", "bf16", 8, 2048, 12, 12, 64), name="attn_train"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "qk", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "scan":
        kind = rng.choice(["step", "fwd", "fwd", "train"])
        D = 8 * _log_int(rng, 8, 512)
        if kind == "step":
            return _scan(kind, dtype, _log_int(rng, 1, 512), 1, D, mix=rng.random() < 0.5)
        T = _log_int(rng, 1, min(65536, (32 << 20) // D))
        most = max(1, min(64, (16 << 20) // (T * D)))
        if rng.random() < 0.4:
            T = min(T * most, 65536)
            return _scan(kind, dtype, 1, T, D, packed=rng.randint(1, min(T, 40)), mix=rng.random() < 0.5)
        return _scan(kind, dtype, rng.randint(1, most), T, D, mix=rng.random() < 0.5)
    d = rng.choice([32, 64, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 8])
    if op == "qk":
        return _qk(rng.choice(["fwd", "fwd", "bwd"]), dtype, _log_int(rng, 1, 16384), hq, hk, d,
                   16 * rng.randint(1, d // 16), rng.choice(["half", "interleaved"]), _log_int(rng, 64, 1 << 20),
                   up=rng.choice(["same", "fp32"]))
    kind = rng.choice(["fwd", "fwd", "train", "token"])
    n = _log_int(rng, 1, 32)
    if kind == "token":
        return _attn("fwd", dtype, n, 1, hq, hk, d, ragged=True, prefix=_log_int(rng, 16, 16384))
    # at most 2^30 scores over the padded batch
    lq = _log_int(rng, 1, int(math.sqrt((1 << 30) / (n * hq))))
    prefix = rng.choice([0, 0, _log_int(rng, 1, max(1, lq // 2))])
    return _attn(kind, dtype, n, lq, hq, hk, d, ragged=rng.random() < 0.7, prefix=prefix)


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------

def _cuts(total, n):
    """n sequence lengths >= 1 that add up to total, the same for every seed."""
    r = random.Random(total * 1009 + n)
    at = sorted(r.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + at, at + [total])]


def _lens(case):
    """(query lengths, key lengths) of an attention case."""
    n, lq, prefix = case["n"], case["lq"], case["prefix"]
    r = random.Random(n * 7919 + lq * 31 + prefix)
    q = [r.randint(max(1, lq // 4), lq) if case["ragged"] else lq for _ in range(n)]
    p = [r.randint(prefix // 4, prefix) if case["ragged"] else prefix for _ in range(n)]
    q[0], p[0] = lq, prefix
    return q, [a + b for a, b in zip(q, p)]


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

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = dict(case=case)
    if case["op"] == "scan":
        B, T, D = case["B"], case["T"], case["D"]
        shape = (B, D) if case["kind"] == "step" else (T, D) if case["packed"] else (B, T, D)
        n = case["packed"] or B
        s["x"] = normal(*shape, dtype=dt)
        # decays as the benchmark's softplus recipe: most of them within 0.1 of 1
        s["g"] = (-torch.nn.functional.softplus(normal(*shape)) * 0.1).to(dt)
        s["init"] = normal(n, D)
        if case["packed"]:
            s["lens"] = _cuts(T, n)
            s["cu"] = _offsets(s["lens"], dev)
        if case["kind"] == "train":
            s["dh"], s["dfinal"] = normal(*shape, dtype=dt), normal(n, D)
    elif case["op"] == "qk":
        N, hq, hk, d, rot = case["tokens"], case["hq"], case["hk"], case["d"], case["rot"]
        s["q"], s["k"] = normal(N, hq, d, dtype=dt), normal(N, hk, d, dtype=dt)
        s["wq"], s["wk"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
        s["pos"] = torch.randint(0, case["far"], (N,), generator=g, device=dev, dtype=torch.int32)
        j = torch.arange(rot // 2, device=dev, dtype=torch.float64)
        s["freq"] = 10000.0 ** (-2 * j / rot)
        if case["kind"] == "bwd":
            up = torch.float32 if case["up"] == "fp32" else dt
            s["dq"], s["dk"] = normal(N, hq, d, dtype=up), normal(N, hk, d, dtype=up)
    else:
        ql, kl = _lens(case)
        s["ql"], s["kl"] = ql, kl
        s["cuq"], s["cuk"] = _offsets(ql, dev), _offsets(kl, dev)
        hq, hk, d = case["hq"], case["hk"], case["d"]
        s["q"], s["k"] = normal(sum(ql), hq, d, dtype=dt), normal(sum(kl), hk, d, dtype=dt)
        s["v"] = normal(sum(kl), hk, d, dtype=dt)
        if case["kind"] == "train":
            s["do"] = normal(sum(ql), hq, d, dtype=dt)
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "scan":
        n = case["B"] * case["T"] * case["D"]
        st = 4 * case["D"] * (case["packed"] or case["B"])
        if case["kind"] == "train":   # x, g, dh in; h, dx, dg out (x and g once for each direction)
            return dict(bytes=8 * n * e + 4 * st, flops=16 * n)
        return dict(bytes=3 * n * e + 2 * st, flops=6 * n)
    if case["op"] == "qk":
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["d"]
        if case["kind"] == "bwd":
            return dict(bytes=n * (2 * e + (4 if case["up"] == "fp32" else e)) + 4 * case["tokens"], flops=16 * n)
        return dict(bytes=2 * n * e + 4 * case["tokens"], flops=8 * n)
    ql, kl = _lens(case)
    d, hq, hk = case["d"], case["hq"], case["hk"]
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(ql, kl))   # causal from the end, key length >= query length
    nq, nk = sum(ql) * hq * d, sum(kl) * hk * d
    if case["kind"] == "train":   # both directions: q, k, v, do, o in; o, dq, dk, dv out
        return dict(bytes=e * (6 * nq + 6 * nk) + 8 * sum(ql) * hq, flops=14 * pairs * d * hq)
    return dict(bytes=e * (2 * nq + 2 * nk) + 4 * sum(ql) * hq, flops=4 * pairs * d * hq)


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------

def run(s):
    return dict(scan=_run_scan, qk=_run_qk, attn=_run_attn)[s["case"]["op"]](s)


def _doubling(a, u):
    """h_t = a_t h_{t-1} + u_t along dim -2 from h = 0, by doubling spans."""
    k = 1
    while k < u.shape[-2]:
        u = torch.cat([u[..., :k, :], u[..., k:, :] + a[..., k:, :] * u[..., :-k, :]], -2)
        a = torch.cat([a[..., :k, :], a[..., k:, :] * a[..., :-k, :]], -2)
        k *= 2
    return u


def _run_scan(s):
    c = s["case"]
    if own:
        import recurrent_sequence_models_amd as rsm
        if c["kind"] == "step":
            state = s["init"].clone()
            return dict(h=rsm.gated_scan_step(s["x"], s["g"], state, mix=c["mix"]), final=state)
        train = c["kind"] == "train"
        h, final, states = rsm.gated_scan(s["x"], s["g"], cu_seqlens=s.get("cu"), mix=c["mix"], init=s["init"],
                                          chunk_states=train)
        if not train:
            return dict(h=h, final=final)
        gr = rsm.gated_scan_bwd(s["x"], s["g"], s["dh"], states, cu_seqlens=s.get("cu"), mix=c["mix"],
                                init=s["init"], d_final=s["dfinal"])
        return dict(h=h, final=final, dx=gr["dx"], dg=gr["dg"], dinit=gr["d_init"])
    dt = s["x"].dtype
    x, g = s["x"].float(), s["g"].float()
    lam = torch.exp(g)
    w = -torch.expm1(g) if c["mix"] else None
    u = x * w if c["mix"] else x
    if c["kind"] == "step":
        h = lam * s["init"] + u
        return dict(h=h.to(dt), final=h)
    # first[n], last[n]: where sequence n begins and ends on the flattened time axis of each batch row
    if c["packed"]:
        first, last = s["cu"][:-1].long(), s["cu"][1:].long() - 1
        a, b = lam.clone(), u.clone()
        a[first] = 0
        b[first] += lam[first] * s["init"]
    else:
        a, b = lam.clone(), u.clone()
        a[:, 0] = 0
        b[:, 0] += lam[:, 0] * s["init"]
    h = _doubling(a, b)
    final = h[last] if c["packed"] else h[:, -1].clone()
    if c["kind"] != "train":
        return dict(h=h.to(dt), final=final)
    # delta_t = dh_t + lam_{t+1} delta_{t+1}, from the right; d_final enters at each sequence's last step
    d = s["dh"].float()
    prev = torch.cat([torch.zeros_like(h[..., :1, :]), h[..., :-1, :]], -2)
    if c["packed"]:
        d[last] += s["dfinal"]
        prev[first] = s["init"]
    else:
        d[:, -1] += s["dfinal"]
        prev[:, 0] = s["init"]
    nxt = torch.cat([a[..., 1:, :], torch.zeros_like(a[..., :1, :])], -2)
    delta = torch.flip(_doubling(torch.flip(nxt, [-2]), torch.flip(d, [-2])), [-2])
    r = lam * delta
    dx, dg = (delta * w, r * (prev - x)) if c["mix"] else (delta, r * prev)
    return dict(h=h.to(dt), final=final, dx=dx.to(dt), dg=dg.to(dt), dinit=r[first] if c["packed"] else r[:, 0].clone())


def _rotate(x, cos, sin, rot, layout, back=False):
    """The first `rot` of the last dim turned by the angles (back: by their negatives)."""
    if back:
        sin = -sin
    a, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        p, q = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat([p * cos - q * sin, q * cos + p * sin], -1)
    else:
        p, q = a[..., 0::2], a[..., 1::2]
        y = torch.stack([p * cos - q * sin, q * cos + p * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _qk_plain(s, x, w, dy, cos, sin):
    c = s["case"]
    dt, xf = x.dtype, x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
    if dy is None:
        return _rotate(xf * r * w, cos, sin, c["rot"], c["layout"]).to(dt)
    u = _rotate(dy.float(), cos, sin, c["rot"], c["layout"], back=True)
    xr = xf * r
    dw = (u * xr).sum((0, 1), dtype=torch.float64).float()
    wu = w * u
    return (r * (wu - xr * (wu * xr).mean(-1, keepdim=True))).to(dt), dw


def _run_qk(s):
    c = s["case"]
    if own:
        import recurrent_sequence_models_amd as rsm
        if c["kind"] == "bwd":
            gr = rsm.qk_norm_rope_bwd(s["q"], s["k"], s["pos"], s["freq"], s["dq"], s["dk"], q_weight=s["wq"],
                                      k_weight=s["wk"], layout=c["layout"])
            return dict(dq=gr["dq"], dk=gr["dk"], dwq=gr["dq_weight"], dwk=gr["dk_weight"])
        q, k = rsm.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["wq"], k_weight=s["wk"],
                                layout=c["layout"])
        return dict(q=q, k=k)
    ang = s["pos"].double()[:, None] * s["freq"]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if c["kind"] == "bwd":
        dq, dwq = _qk_plain(s, s["q"], s["wq"], s["dq"], cos, sin)
        dk, dwk = _qk_plain(s, s["k"], s["wk"], s["dk"], cos, sin)
        return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    return dict(q=_qk_plain(s, s["q"], s["wq"], None, cos, sin), k=_qk_plain(s, s["k"], s["wk"], None, cos, sin))


def _padded(x, cu, most):
    """[total, H, d] to [N, H, most, d], zeros past each sequence's end, and the rows' validity."""
    at = cu[:-1].long()[:, None] + torch.arange(most, device=x.device)
    ok = torch.arange(most, device=x.device) < (cu[1:] - cu[:-1]).long()[:, None]
    y = torch.where(ok[..., None, None], x[at.clamp(max=x.shape[0] - 1)].float(), torch.zeros((), device=x.device))
    return y.transpose(1, 2).contiguous(), ok


def _run_attn(s):
    c = s["case"]
    if own:
        import recurrent_sequence_models_amd as rsm
        o, lse = rsm.attention_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cuq"], cu_seqlens_k=s["cuk"])
        if c["kind"] != "train":
            return dict(o=o, lse=lse)
        gr = rsm.attention_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], cu_seqlens=s["cuq"], cu_seqlens_k=s["cuk"])
        return dict(o=o, lse=lse, dq=gr["dq"], dk=gr["dk"], dv=gr["dv"])
    dt, dev = s["q"].dtype, s["q"].device
    n, hq, hk, d = c["n"], c["hq"], c["hk"], c["d"]
    grp, mq, mk = hq // hk, max(s["ql"]), max(s["kl"])
    scale = d ** -0.5
    q, okq = _padded(s["q"], s["cuq"], mq)
    k, okk = _padded(s["k"], s["cuk"], mk)
    v, _ = _padded(s["v"], s["cuk"], mk)
    # the query heads of a key head side by side: [N, hk, grp * mq, d]
    q = q.view(n, hk, grp * mq, d)
    lq, lk = (s["cuq"][1:] - s["cuq"][:-1]).long(), (s["cuk"][1:] - s["cuk"][:-1]).long()
    row = torch.arange(mq, device=dev)[:, None] + (lk - lq)[:, None, None]
    see = (torch.arange(mk, device=dev) <= row) & okk[:, None]
    see = see[:, None, None]                                       # [N, 1, 1, mq, mk]
    t = torch.matmul(q, k.transpose(2, 3)).view(n, hk, grp, mq, mk) * scale
    t = t.masked_fill(~see, -math.inf)
    top = t.amax(-1, keepdim=True).clamp(min=-1e30)
    t = torch.exp(t - top)
    total = t.sum(-1, keepdim=True)
    p = (t / total).view(n, hk, grp * mq, mk)
    lse = (top + torch.log(total)).view(n, hq, mq)
    o = torch.matmul(p, v)

    def packed(x, ok, heads, length):
        return x.reshape(n, heads, length, d).transpose(1, 2)[ok].to(dt)

    out = dict(o=packed(o, okq, hq, mq), lse=lse.transpose(1, 2)[okq])
    if c["kind"] == "train":
        do, _ = _padded(s["do"], s["cuq"], mq)
        do = do.view(n, hk, grp * mq, d)
        dv = torch.matmul(p.transpose(2, 3), do)
        ds = torch.matmul(do, v.transpose(2, 3))
        ds = p * (ds - (do * o).sum(-1, keepdim=True))
        out.update(dq=packed(torch.matmul(ds, k) * scale, okq, hq, mq),
                   dk=packed(torch.matmul(ds.transpose(2, 3), q) * scale, okk, hk, mk), dv=packed(dv, okk, hk, mk))
    return out


# ---------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return dict(scan=_exact_scan, qk=_exact_qk, attn=_exact_attn)[case["op"]](s)


def _exact_scan(s):
    c = s["case"]
    x, g, h = s["x"].double(), s["g"].double(), s["init"].double()
    lam = g.exp()
    w = -g.expm1() if c["mix"] else torch.ones_like(g)
    if c["kind"] == "step":
        h = lam * h + w * x
        return dict(h=h, final=h)
    T = c["T"]
    begin = {}
    if c["packed"]:   # sequence n begins at begin[t] = n
        at = 0
        for n, length in enumerate(s["lens"]):
            begin[at] = n
            at += length
    time = (lambda y, t: y[t]) if c["packed"] else (lambda y, t: y[:, t])
    hs, prevs = torch.empty_like(x), torch.empty_like(x)
    ends = torch.empty_like(s["init"], dtype=torch.float64)
    state, n = (h if not c["packed"] else None), -1
    for t in range(T):
        if t in begin:
            if n >= 0:
                ends[n] = state
            n, state = begin[t], h[begin[t]]
        time(prevs, t).copy_(state)
        state = time(lam, t) * state + time(w, t) * time(x, t)
        time(hs, t).copy_(state)
    if c["packed"]:
        ends[n] = state
    else:
        ends = state
    out = dict(h=hs, final=ends)
    if c["kind"] == "train":
        dh, dfin = s["dh"].double(), s["dfinal"].double()
        dx, dg, dinit = torch.empty_like(x), torch.empty_like(x), torch.empty_like(ends)
        r = dfin if not c["packed"] else dfin[n]
        for t in range(T - 1, -1, -1):
            delta = time(dh, t) + r
            r = time(lam, t) * delta
            time(dx, t).copy_(delta * time(w, t))
            # d lam / d g = lam; in the mixed form the input's weight falls as lam grows
            time(dg, t).copy_(r * (time(prevs, t) - time(x, t)) if c["mix"] else r * time(prevs, t))
            if t in begin:
                dinit[begin[t]] = r
                r = dfin[begin[t] - 1]
        if not c["packed"]:
            dinit = r
        out.update(dx=dx, dg=dg, dinit=dinit)
    return out


def _exact_qk(s):
    c = s["case"]
    half = c["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["pos"].double()[:, None] * s["freq"])[:, None]           # e^{i angle}
    i = torch.arange(half, device=s["q"].device)
    re, im = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)

    def turned(y, by):
        z = torch.complex(y[..., re], y[..., im]) * by
        y = y.clone()
        y[..., re], y[..., im] = z.real, z.imag
        return y

    out = {}
    for name, x, w in (("q", s["q"].double(), s["wq"].double()), ("k", s["k"].double(), s["wk"].double())):
        ms = x.square().sum(-1, keepdim=True) / c["d"] + 1e-6
        if c["kind"] == "fwd":
            out[name] = turned(w * x / ms.sqrt(), turn)
            continue
        u = turned(s["d" + name].double(), turn.conj())
        out["dw" + name] = (u * x / ms.sqrt()).sum(dim=(0, 1))
        inner = (w * u * x).sum(-1, keepdim=True) / c["d"]
        out["d" + name] = w * u / ms.sqrt() - x * inner / ms ** 1.5
    return out


def _exact_attn(s):
    c = s["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    dev, train = s["q"].device, c["kind"] == "train"
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=dev)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = b = 0
    for lq, lk in zip(s["ql"], s["kl"]):
        hidden = torch.ones(lq, lk, dtype=torch.bool, device=dev).triu(lk - lq + 1)
        for h in range(hq):
            kv = h * hk // hq
            qs, ks, vs = q[a:a + lq, h], k[b:b + lk, kv], v[b:b + lk, kv]
            t = (qs @ ks.T) / math.sqrt(d)
            t[hidden] = -math.inf
            lse[a:a + lq, h] = torch.logsumexp(t, -1)
            p = torch.exp(t - lse[a:a + lq, h, None])
            o[a:a + lq, h] = p @ vs
            if train:
                g = s["do"][a:a + lq, h].double()
                dv[b:b + lk, kv] += p.T @ g
                t = p * (g @ vs.T - (g * o[a:a + lq, h]).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[a:a + lq, h] = t @ ks
                dk[b:b + lk, kv] += t.T @ qs
        a, b = a + lq, b + lk
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv) if train else dict(o=o, lse=lse)
