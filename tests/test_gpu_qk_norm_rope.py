"""GPU parity of the query / key norm with rotary positions (falcon_qk_norm_rope and its
backward) against the fp64 oracle, elementwise.

Bounds, u = 2^-24: a row's root mean square comes from a sum of d squares and one
reciprocal root, 1 / 2 (d + 8) u relative at most; the entries of a pair then take a few
products and sums, and the angle's fraction of a turn is rounded once (2 pi u / 2
absolute) before sine and cosine, which are within 4 u."""

import numpy as np
import pytest

from layer_helpers import U, check, f64, half, rand
from oracle import layer as L

pytestmark = pytest.mark.gpu


def positions(seed, n, far):
    import torch
    p = np.random.Generator(np.random.PCG64(seed)).integers(0, far, size=n)
    return torch.from_numpy(p.astype(np.int32)).cuda()


def turned_bound(z, rot, layout, scale):
    """|z_a| + |z_b| in both places of a pair (times the scale), |z| in the rest."""
    a = np.arange(rot // 2)
    a, b = (a, a + rot // 2) if layout == "half" else (2 * a, 2 * a + 1)
    s = np.abs(z).copy()
    s[..., a] = s[..., b] = (np.abs(z[..., a]) + np.abs(z[..., b])) * abs(scale)
    return s


def run_case(dtype, tokens, hq, hk, d, rot, layout="half", norm=True, weights=True, far=5000, scale=1.0, up="same",
             seed=1, eps=1e-6, base=10000.0):
    import torch
    from recurrent_sequence_models_amd import qk_norm_rope, qk_norm_rope_bwd, rope_frequencies
    q, k = rand(seed, tokens, hq, d, dtype=dtype), rand(seed + 1, tokens, hk, d, dtype=dtype)
    wq, wk = (1 + 0.3 * rand(seed + 2, d), 1 + 0.3 * rand(seed + 3, d)) if weights and norm else (None, None)
    pos = positions(seed + 4, tokens, far)
    freq = rope_frequencies(rot, base, device="cuda")[0] if rot else None
    kw = dict(q_weight=wq, k_weight=wk, norm=norm, eps=eps, layout=layout, rot_scale=scale)
    yq, yk = qk_norm_rope(q, k, pos, freq, **kw)
    gt = "fp32" if up == "fp32" else dtype
    dq, dk = rand(seed + 5, tokens, hq, d, dtype=gt), rand(seed + 6, tokens, hk, d, dtype=gt)
    gr = qk_norm_rope_bwd(q, k, pos, freq, dq, dk, **kw)
    torch.cuda.synchronize()
    F = f64(freq) if rot else np.zeros(0)
    okw = dict(norm=norm, eps=eps, layout=layout, scale=scale)
    ho, c = half(dtype) * (1 + 1e-3), (d + 40) * U
    for name, x, w, y, dy, dx, dw in (("q", q, wq, yq, dq, gr["dq"], gr["dq_weight"]),
                                      ("k", k, wk, yk, dk, gr["dk"], gr["dk_weight"])):
        X, W, P, DY = f64(x), f64(w), f64(pos), f64(dy)
        ref = L.norm_rope(X, W, P, F, **okw)
        z = L.norm_rope(X, W, P, np.zeros(0), **okw)
        check(name, f64(y), ref, c * turned_bound(z, rot, layout, scale) + ho * np.abs(ref))
        rx, rw = L.norm_rope_backward(X, W, P, F, DY, **okw)
        u = turned_bound(DY, rot, layout, scale)            # bounds |u| as well
        r = 1 / np.sqrt(np.mean(X * X, -1, keepdims=True) + eps) if norm else 1.0
        Wn = 1.0 if W is None else np.abs(W)
        inner = Wn * u
        full = r * inner + (np.abs(X) * r ** 3 * np.mean(inner * np.abs(X), -1, keepdims=True) if norm else 0)
        check("d" + name, f64(dx), rx, 4 * c * full + ho * np.abs(rx))
        if w is not None:
            # sums over the rows: a thread's own, its workgroup's and the workgroups', at most
            # rows / 1024 + 600 additions one after the other
            n = X.shape[0] * X.shape[1] / 1024 + 600
            check("dw" + name, f64(dw), rw, (4 * c + n * U) * np.sum(u * np.abs(X) * r, (0, 1)))
        else:
            assert dw is None


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(32, 32), (32, 16), (64, 64), (64, 48), (64, 0), (128, 128), (128, 16), (128, 96),
                                   (128, 112)])
def test_rotations(dtype, layout, d, rot):
    run_case(dtype, 13, 6, 2, d, rot, layout, seed=d + rot)


@pytest.mark.parametrize("dtype,up", [("fp32", "same"), ("bf16", "same"), ("bf16", "fp32")])
@pytest.mark.parametrize("tokens", [1, 2, 63, 4095, 4099])
@pytest.mark.parametrize("hq,hk", [(1, 1), (12, 12), (16, 4), (5, 1)])
def test_tokens_and_heads(dtype, up, tokens, hq, hk):
    """One token, odd counts, and both sizes of a workgroup's share (4 tokens from 4096 on)."""
    run_case(dtype, tokens, hq, hk, 64, 32, "half", up=up, seed=tokens + hq)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_without_norm_or_weights(dtype, layout):
    run_case(dtype, 37, 4, 2, 64, 32, layout, norm=False)
    run_case(dtype, 37, 4, 2, 64, 32, layout, weights=False, scale=1.3)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(layout):
    """Positions up to 2^31 - 1: the angle is formed in 64 bits (2^31 turns of the fastest
    pair leave 2^-22 of one there)."""
    run_case("fp32", 50, 2, 2, 64, 64, layout, far=(1 << 31) - 1, norm=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_zero_rows(dtype):
    """A row of zeros stays zero (eps > 0) and takes r w u as its gradient."""
    import torch
    from recurrent_sequence_models_amd import qk_norm_rope, qk_norm_rope_bwd, rope_frequencies
    q = torch.zeros(3, 2, 64, device="cuda", dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
    pos, f = positions(1, 3, 100), rope_frequencies(64, device="cuda")[0]
    yq, yk = qk_norm_rope(q, q.clone(), pos, f, eps=0.25)
    assert torch.equal(yq, q) and torch.equal(yk, q)
    dy = rand(2, 3, 2, 64, dtype=dtype)
    gr = qk_norm_rope_bwd(q, q.clone(), pos, f, dy, dy.clone(), eps=0.25)
    want, _ = L.norm_rope_backward(f64(q), None, f64(pos), f64(f), f64(dy), eps=0.25)
    check("dq", f64(gr["dq"]), want, 200 * U * 4 * 4 + half(dtype) * np.abs(want))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_views_of_a_projection_and_in_place(dtype):
    """q and k as views of one [B, T, (hq + 2 hk) d] output, results written over them, and
    gradients written into a view; the values beside them stay."""
    import torch
    from recurrent_sequence_models_amd import qk_norm_rope, qk_norm_rope_bwd, rope_frequencies
    B, T, hq, hk, d = 2, 70, 6, 2, 64
    qkv = rand(1, B, T, hq + 2 * hk, d, dtype=dtype)
    f = rope_frequencies(32, device="cuda")[0]
    pos = positions(2, B * T, 900).view(B, T)
    dense = qk_norm_rope(qkv[:, :, :hq].contiguous(), qkv[:, :, hq:hq + hk].contiguous(), pos, f)
    keep = qkv.clone()
    got = qk_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hk], pos, f)
    assert torch.equal(got[0], dense[0]) and torch.equal(got[1], dense[1]) and torch.equal(qkv, keep)
    dq, dk = rand(3, B, T, hq, d), rand(4, B, T, hk, d)
    w = 1 + 0.1 * rand(5, d)
    a = qk_norm_rope_bwd(keep[:, :, :hq].contiguous(), keep[:, :, hq:hq + hk].contiguous(), pos, f, dq, dk, q_weight=w,
                         k_weight=w)
    grad = torch.full_like(qkv, 3.0)
    b = qk_norm_rope_bwd(keep[:, :, :hq], keep[:, :, hq:hq + hk], pos, f, dq, dk, q_weight=w, k_weight=w,
                         out=dict(dq=grad[:, :, :hq], dk=grad[:, :, hq:hq + hk]))
    assert torch.equal(grad[:, :, :hq], a["dq"]) and torch.equal(grad[:, :, hq:hq + hk], a["dk"])
    assert torch.all(grad[:, :, hq + hk:] == 3.0) and torch.equal(a["dq_weight"], b["dq_weight"])
    qk_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hk], pos, f, out=(qkv[:, :, :hq], qkv[:, :, hq:hq + hk]))
    assert torch.equal(qkv[:, :, :hq], dense[0]) and torch.equal(qkv[:, :, hq:hq + hk], dense[1])
    assert torch.equal(qkv[:, :, hq + hk:], keep[:, :, hq + hk:])


def test_streams_and_graph():
    import torch
    from recurrent_sequence_models_amd import qk_norm_rope, qk_norm_rope_bwd, rope_frequencies
    q, k = rand(1, 300, 4, 64, dtype="bf16"), rand(2, 300, 2, 64, dtype="bf16")
    w = 1 + 0.1 * rand(3, 64)
    pos, f = positions(4, 300, 5000), rope_frequencies(64, device="cuda")[0]

    def call(**kw):
        y = qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w, **kw)
        g = qk_norm_rope_bwd(q, k, pos, f, y[0], y[1], q_weight=w, k_weight=w, **kw)
        return [*y, g["dq"], g["dk"], g["dq_weight"], g["dk_weight"]]

    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    import torch
    from recurrent_sequence_models_amd import FalconError, qk_norm_rope, qk_norm_rope_bwd, rope_frequencies
    q, k = rand(1, 8, 4, 64), rand(2, 8, 2, 64)
    pos, f = positions(3, 8, 10), rope_frequencies(64, device="cuda")[0]
    bad = [
        (TypeError, lambda: qk_norm_rope(q.half(), k.half(), pos, f)),
        (TypeError, lambda: qk_norm_rope(q, k.bfloat16(), pos, f)),
        (TypeError, lambda: qk_norm_rope(q, k, pos.long(), f)),
        (TypeError, lambda: qk_norm_rope(q, k, pos, f.float())),
        (ValueError, lambda: qk_norm_rope(q, k[:4], pos, f)),
        (ValueError, lambda: qk_norm_rope(q, k, pos[:4], f)),
        (ValueError, lambda: qk_norm_rope(q, k, pos, f, layout="other")),
        (ValueError, lambda: qk_norm_rope(q, k, pos, f, q_weight=torch.ones(32, device="cuda"))),
        (ValueError, lambda: qk_norm_rope(q, k, pos, f, norm=False, q_weight=torch.ones(64, device="cuda"))),
        (ValueError, lambda: qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2), pos, f)),
        (ValueError, lambda: qk_norm_rope(q[:, :, ::2], k[:, :, ::2], pos, f)),
        (ValueError, lambda: qk_norm_rope(q[:, ::2], k, pos, f)),
        (ValueError, lambda: qk_norm_rope(q[:1].expand(8, 4, 64), k, pos, f)),
        (FalconError, lambda: qk_norm_rope(q[..., :48].contiguous(), k[..., :48].contiguous(), pos, f[:16])),
        (FalconError, lambda: qk_norm_rope(q, k, pos, f[:12])),      # rot = 24, not a multiple of 16
        (FalconError, lambda: qk_norm_rope(q, k, pos, torch.cat([f, f]))),   # rot = 128 > d
        (FalconError, lambda: qk_norm_rope(q, k, pos, f, eps=-1.0)),
        (FalconError, lambda: qk_norm_rope(q, k, pos, f, rot_scale=float("nan"))),
        (FalconError, lambda: qk_norm_rope(q, k, pos, f, out=(rand(5, 8, 4, 66)[..., 1:65], k))),   # distances not 16 bytes
        (TypeError, lambda: qk_norm_rope_bwd(q, k, pos, f, q, k.bfloat16())),
        (FalconError, lambda: qk_norm_rope_bwd(q, k, pos, f, q.bfloat16(), k.bfloat16())),   # fp32 inputs, bf16 gradients
        (ValueError, lambda: qk_norm_rope(q.cpu(), k.cpu(), pos, f)),
    ]
    for i, (err, f_) in enumerate(bad):
        with pytest.raises((err, ValueError) if err is FalconError else err):
            f_()
            raise AssertionError(f"call {i} was taken")


def test_more_tokens_than_a_launch_of_one_group_each():
    """2^26 tokens and some: workgroups come round again, and the last tokens are as in a short call."""
    import torch
    from recurrent_sequence_models_amd import qk_norm_rope, rope_frequencies
    n, tail, d = (1 << 26) + 5, 4099, 32
    freq, _ = rope_frequencies(d, device="cuda")
    q = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros_like(q)
    at = [slice(0, tail), slice((1 << 20) - 7, (1 << 20) + tail), slice(n - tail, n)]   # 2^18 groups of 4 tokens in a round
    for i, s in enumerate(at):
        q[s] = rand(2 * i, s.stop - s.start, 1, d, dtype="bf16")
        k[s] = rand(2 * i + 1, s.stop - s.start, 1, d, dtype="bf16")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    want = [qk_norm_rope(q[s], k[s], pos[s], freq) for s in at]
    qk_norm_rope(q, k, pos, freq, out=(q, k))
    for s, (wq, wk) in zip(at, want):
        assert torch.equal(q[s], wq) and torch.equal(k[s], wk)
    assert not q[tail:(1 << 20) - 7].any()


def test_numbers_in_changing_tensors():
    """eps and the scale are taken by their value at the call, whatever object holds them."""
    import torch
    from recurrent_sequence_models_amd import qk_norm_rope, rope_frequencies
    q, pos = rand(1, 9, 2, 64), torch.arange(9, dtype=torch.int32, device="cuda")
    freq, _ = rope_frequencies(64, device="cuda")
    eps, scale = torch.tensor(1e-6), torch.tensor(1.0)
    a = qk_norm_rope(q, q, pos, freq, eps=eps, rot_scale=scale)[0]
    eps.fill_(0.5), scale.fill_(2.0)
    b = qk_norm_rope(q, q, pos, freq, eps=eps, rot_scale=scale)[0]
    assert torch.equal(a, qk_norm_rope(q, q, pos, freq)[0])
    assert torch.equal(b, qk_norm_rope(q, q, pos, freq, eps=0.5, rot_scale=2.0)[0])
