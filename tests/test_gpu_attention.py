"""GPU parity of causal attention (falcon_attn_fwd, falcon_attn_bwd) against the fp64
oracle, elementwise, with the bounds of layer_helpers.attention_bounds."""

import numpy as np
import pytest

from layer_helpers import attention_bounds, check, f64, offsets, rand
from oracle import layer as L

pytestmark = pytest.mark.gpu


def run_case(dtype, ql, kl, hq, hk, d, packed=True, scale=None, seed=1, back=True, behind=0, spread=1.0):
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    nq, nk = sum(ql) + behind, sum(kl) + behind
    q, do = rand(seed, nq, hq, d, dtype=dtype, scale=spread), rand(seed + 3, nq, hq, d, dtype=dtype)
    k, v = rand(seed + 1, nk, hk, d, dtype=dtype, scale=spread), rand(seed + 2, nk, hk, d, dtype=dtype)
    if packed:
        kw = dict(cu_seqlens=offsets(ql), cu_seqlens_k=offsets(kl), scale=scale)
        args = (q, k, v)
    else:
        kw = dict(scale=scale)
        args = (q.view(len(ql), ql[0], hq, d), k.view(len(kl), kl[0], hk, d), v.view(len(kl), kl[0], hk, d))
    out = torch.full_like(args[0], 7.0)
    o, lse = attention_fwd(*args, out=out, **kw)
    grads = None
    if back:
        grads = attention_bwd(*args, o, lse, do.view(o.shape), **kw,
                              out=dict(dq=torch.full_like(args[0], 7.0), dk=torch.full_like(args[1], 7.0),
                                       dv=torch.full_like(args[2], 7.0)))
        grads = {n: f64(t).reshape(-1, *t.shape[-2:]) for n, t in grads.items()}
    torch.cuda.synchronize()
    O, LSE = f64(o).reshape(nq, hq, d), f64(lse).reshape(nq, hq)
    Q, K, V, DO = f64(q), f64(k), f64(v), f64(do)
    sc = float(np.float32(d ** -0.5 if scale is None else scale))
    for i, ((a, b), (c, e)) in enumerate(zip(L.ranges(ql), L.ranges(kl))):
        if b == a and e == c:
            continue
        ref = attention_bounds(Q[a:b], K[c:e], V[c:e], sc, dtype, DO[a:b] if back else None)
        check(f"o[{i}]", O[a:b], ref["o"], ref["bo"])
        none = np.isneginf(ref["lse"])
        assert np.all(np.isneginf(LSE[a:b]) == none) and np.all(O[a:b][none] == 0), i
        check(f"lse[{i}]", np.where(none, 0, LSE[a:b]), np.where(none, 0, ref["lse"]), ref["bl"])
        if back:
            for n, lo, hi, bn in (("dq", a, b, "bq"), ("dk", c, e, "bk"), ("dv", c, e, "bv")):
                check(f"{n}[{i}]", grads[n][lo:hi], ref[n], ref[bn] * 1.01)
    if behind:
        assert np.all(O[-behind:] == 7.0)
        if back:
            assert all(np.all(g[-behind:] == 7.0) for g in grads.values())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 129])
def test_lengths(dtype, d, T):
    run_case(dtype, [T, T], [T, T], 2, 2, d, packed=False, seed=T + d)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (4, 2), (8, 1), (5, 5), (12, 2), (40, 1)])
def test_groups(dtype, hq, hk):
    """Groups that do and do not divide a tile's rows."""
    run_case(dtype, [50, 7], [50, 7], hq, hk, 64, seed=hq)


PACKED = [([1], [1]), ([5, 0, 70, 1, 1], [5, 0, 70, 1, 1]), ([3, 40, 1, 0], [90, 40, 130, 6]),
          ([1, 1, 1, 1], [200, 1, 64, 65]), ([10, 5], [4, 0]), ([64, 128, 1], [64, 128, 1]), ([0, 0, 9], [3, 0, 9])]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", PACKED, ids=lambda p: "q" + "-".join(map(str, p[0])))
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (3, 3, 128)])
def test_packed(dtype, lens, hq, hk, d):
    """Ragged and empty sequences, keys before the queries, more queries than keys (rows
    that see nothing: o = 0, lse = -inf, no gradients)."""
    run_case(dtype, *lens, hq, hk, d, seed=sum(lens[0]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_leaves_the_rest(dtype):
    run_case(dtype, [40, 0, 33], [40, 0, 33], 4, 2, 64, behind=9)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [([1], [1500]), ([1, 1, 0, 1], [3000, 1, 5, 700]), ([2, 3], [1111, 2048]),
                                  ([40], [1300])], ids=["one", "ragged", "few", "rows"])
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (2, 2, 64), (6, 2, 32), (40, 1, 64)])
def test_split_keys(dtype, lens, hq, hk, d):
    """Few queries against many keys: the keys are split over workgroups and joined."""
    run_case(dtype, *lens, hq, hk, d, back=False, seed=hq + d)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_scores_and_scale(dtype):
    """Peaked rows (scores of several hundred) and a scale of the caller's."""
    run_case(dtype, [70], [70], 2, 1, 64, scale=0.5, spread=3.0, seed=3)


def test_longer_prompt():
    """A few thousand tokens: running maxima over many tiles, several row and key tiles."""
    run_case("bf16", [1100], [1100], 2, 1, 64, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_views_and_other_sequences(dtype):
    """q, k, v as views of one projection; NaN in the sequences beside and behind one do not
    reach it; gradients into views leave the rest."""
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    hq, hk, d, lens = 4, 2, 64, [30, 45, 20]
    qkv = rand(1, sum(lens) + 3, hq + 2 * hk, d, dtype=dtype)
    do = rand(2, sum(lens) + 3, hq, d, dtype=dtype)
    cu = offsets(lens)
    cut = lambda t: (t[:, :hq], t[:, hq:hq + hk], t[:, hq + hk:])  # noqa: E731
    dense = [t.contiguous() for t in cut(qkv)]
    o, lse = attention_fwd(*dense, cu_seqlens=cu)
    g = attention_bwd(*dense, o, lse, do, cu_seqlens=cu)
    bad = qkv.clone()
    bad[:30], bad[75:] = float("nan"), float("inf")
    bad_do = do.clone()
    bad_do[:30], bad_do[75:] = float("inf"), float("nan")
    o2, lse2 = attention_fwd(*cut(bad), cu_seqlens=cu)
    grad = torch.full_like(qkv, 3.0)
    attention_bwd(*cut(bad), o2, lse2, bad_do, cu_seqlens=cu, out=dict(zip(("dq", "dk", "dv"), cut(grad))))
    s = slice(30, 75)
    assert torch.equal(o[s], o2[s]) and torch.equal(lse[s], lse2[s])
    for n, t in zip(("dq", "dk", "dv"), cut(grad)):
        assert torch.equal(g[n][s], t[s])
    assert torch.all(grad[-3:] == 3.0)


def test_streams_and_graph():
    """Another stream, and a captured forward and backward (split keys too), replayed."""
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    q, k, v = (rand(i, 2, 150, h, 64, dtype="bf16") for i, h in ((1, 4), (2, 2), (3, 2)))
    t, kk, vv = rand(4, 2, 1, 4, 64, dtype="bf16"), rand(5, 2, 2000, 2, 64, dtype="bf16"), rand(6, 2, 2000, 2, 64, dtype="bf16")

    def call(**kw):
        o, lse = attention_fwd(q, k, v, **kw)
        g = attention_bwd(q, k, v, o, lse, o, **kw)
        return [o, lse, g["dq"], g["dk"], g["dv"], *attention_fwd(t, kk, vv, **kw)]

    want = call()
    torch.cuda.synchronize()
    got = call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    import torch
    from recurrent_sequence_models_amd import FalconError, attention_bwd, attention_fwd
    q, k = rand(1, 2, 16, 4, 64), rand(2, 2, 16, 2, 64)
    o, lse = attention_fwd(q, k, k)
    bad = [
        (TypeError, lambda: attention_fwd(q.half(), k.half(), k.half())),
        (TypeError, lambda: attention_fwd(q, k, k.bfloat16())),
        (ValueError, lambda: attention_fwd(q, k, k[:, :8])),
        (ValueError, lambda: attention_fwd(q[0], k[0], k[0])),
        (ValueError, lambda: attention_fwd(q, k, k, cu_seqlens=offsets([16, 16]))),
        (ValueError, lambda: attention_fwd(q[0], k[0], k[0], cu_seqlens=offsets([16]), cu_seqlens_k=offsets([8, 8]))),
        (ValueError, lambda: attention_fwd(q[0], k[0, :8], k[0, :8], cu_seqlens=offsets([16]))),
        (ValueError, lambda: attention_fwd(q.transpose(1, 2), k.transpose(1, 2), k.transpose(1, 2))),
        (FalconError, lambda: attention_fwd(q[:, :, :3].contiguous(), k, k)),          # 3 heads over 2
        (FalconError, lambda: attention_fwd(q[..., :48].contiguous(), k[..., :48].contiguous(), k[..., :48].contiguous())),
        (FalconError, lambda: attention_fwd(q, k, k, scale=0.0)),
        (FalconError, lambda: attention_fwd(q, k, k, scale=float("inf"))),
        (FalconError, lambda: attention_fwd(rand(1, 1, 1, 1, 64), rand(2, 1, 4000, 1, 64), rand(3, 1, 4000, 1, 64),
                                            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: attention_bwd(q, k, k, o, lse[:, :8], o)),
        (TypeError, lambda: attention_bwd(q, k, k, o, lse, o.bfloat16())),
        (ValueError, lambda: attention_fwd(q.cpu(), k.cpu(), k.cpu())),
    ]
    for i, (err, f_) in enumerate(bad):
        with pytest.raises(err):
            f_()
            raise AssertionError(f"call {i} was taken")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ql,kl,hq,hk,d", [([200], [200], 2, 2, 64), ([130], [170], 4, 1, 128), ([40], [40], 3, 1, 32),
                                           ([4], [90], 2, 1, 64), ([3], [1500], 4, 2, 128), ([70, 60], [70, 61], 2, 1, 64)])
def test_keys_behind_the_mask(dtype, ql, kl, hq, hk, d):
    """Infinite and NaN keys and values do not reach the queries that do not see them, and do
    reach those that see them (split keys too)."""
    import torch
    from recurrent_sequence_models_amd import attention_fwd
    q, k, v = rand(1, sum(ql), hq, d, dtype=dtype), rand(2, sum(kl), hk, d, dtype=dtype), rand(3, sum(kl), hk, d, dtype=dtype)
    kw = dict(cu_seqlens=offsets(ql), cu_seqlens_k=offsets(kl))
    o, lse = attention_fwd(q, k, v, **kw)
    for back in (1, 2, min(ql[0] - 1, 37)):                # the bad key: so many from the first sequence's end
        j = kl[0] - back
        i = ql[0] - back                                   # the first query that sees it
        for name, bad in (("nan", (float("nan"),) * d), ("inf", (float("inf"), -float("inf")) * (d // 2))):
            v2 = v.clone()
            v2[j, :] = torch.tensor(bad, device="cuda").to(v.dtype)
            o2, lse2 = attention_fwd(q, k, v2, **kw)
            keep = torch.ones(sum(ql), dtype=torch.bool, device="cuda")
            keep[i:ql[0]] = False
            assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2, lse), (name, back)
            seen = o2[~keep].float()
            assert torch.isnan(seen).all() if name == "nan" else torch.equal(seen, v2[j].float().repeat_interleave(
                hq // hk, 0).expand_as(seen)), (name, back)
        k2 = k.clone()
        k2[j] = float("nan")
        o2, lse2 = attention_fwd(q, k2, v, **kw)
        assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])
        assert torch.isnan(o2[~keep].float()).all() and torch.isnan(lse2[~keep]).all()
        v2[j], v2[j - 1] = float("inf"), -float("inf")     # both: NaN where both are seen
        o2, _ = attention_fwd(q, k, v2, **kw)
        assert torch.isnan(o2[i:ql[0]].float()).all()
        if i > 0:
            assert torch.all(o2[i - 1].float() == -float("inf"))


@pytest.mark.parametrize("d", [64, 128])
def test_widest_strides(d):
    """Tokens 2^25 bytes apart, the widest there are."""
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    T, step = 131, 1 << 23
    wide = torch.empty(T, step, device="cuda")
    parts = [rand(i, T, 2, d) for i in range(4)]
    views = []
    for i, t in enumerate(parts):
        v = wide[:, i * step // 4:][:, :2 * d].unflatten(1, (2, d))
        v.copy_(t)
        views.append(v)
    cu = offsets([T])
    (q, k, v, do), (wq, wk, wv, wdo) = parts, views
    o, lse = attention_fwd(q, k, v, cu_seqlens=cu)
    o2, lse2 = attention_fwd(wq, wk, wv, cu_seqlens=cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    want = attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu)
    got = attention_bwd(wq, wk, wv, o, lse, wdo, cu_seqlens=cu, out=None)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(want[n], got[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [([1], [20000]), ([1, 1], [40000, 3]), ([1, 0, 2, 3], [9000, 7, 1, 20001]),
                                  ([5] * 40, [1100] * 40)], ids=["one", "uneven", "mixed", "few"])
def test_many_splits(dtype, lens):
    """Up to 128 splits of the keys, most of them empty for the short sequences; and few, of many rows."""
    run_case(dtype, *lens, 4, 1, 64, back=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ql,kl,hq,hk,d", [([1], [1], 2, 2, 64), ([1], [33], 2, 1, 128), ([1, 1], [33, 40], 4, 1, 32),
                                           ([1], [1500], 4, 2, 64), ([1, 1], [20001, 70], 4, 1, 128),
                                           ([129], [129], 2, 2, 64), ([129, 1], [129, 1], 1, 1, 128), ([257], [300], 1, 1, 32)])
def test_infinite_value_at_the_end(dtype, ql, kl, hq, hk, d):
    """An infinite value of the last key, where a tile of keys ends behind it: inf for the query
    that sees it (the last one), however many keys there are, and nothing for the others."""
    import torch
    from recurrent_sequence_models_amd import attention_fwd
    q, k, v = rand(1, sum(ql), hq, d, dtype=dtype), rand(2, sum(kl), hk, d, dtype=dtype), rand(3, sum(kl), hk, d, dtype=dtype)
    kw = dict(cu_seqlens=offsets(ql), cu_seqlens_k=offsets(kl))
    o, lse = attention_fwd(q, k, v, **kw)
    v2 = v.clone()
    j, i = kl[0] - 1, ql[0] - 1
    v2[j, :, ::2], v2[j, :, 1::4] = float("inf"), -float("inf")     # every fourth entry stays as it is
    o2, lse2 = attention_fwd(q, k, v2, **kw)
    keep = torch.ones(sum(ql), dtype=torch.bool, device="cuda")
    keep[i] = False
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2, lse)
    want = torch.where(torch.isfinite(v2[j]), torch.zeros_like(v2[j]), v2[j]).repeat_interleave(hq // hk, 0)
    assert torch.equal(o2[i], o[i] + want)


def splits(nq, nk, n, hq, hk, d, dtype, back, packed=True):
    """How many workgroups share the keys of a forward (the rows of a backward) of nq query and
    nk key tokens, from the partial results that its workspace holds."""
    import ctypes
    from recurrent_sequence_models_amd.falcon import AttnShape, lib
    tq, tk = (nq, nk) if packed else (nq // n, nk // n)
    s = AttnShape(1 if dtype == "bf16" else 0, n, tq, tk, hq, hk, d, 1.0)
    if not back:
        return max(lib().falcon_attn_fwd_workspace(ctypes.byref(s), packed) // (nq * hq * (d + 2) * 4), 1)
    rows = 2 * (-(-nq * hq * 4 // 16) * 16)
    return max((lib().falcon_attn_bwd_workspace(ctypes.byref(s), packed) - rows) // (2 * nk * hk * d * 4), 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ql,kl,least,behind", [([1], [20000], 65, 0), ([1, 0, 1, 2], [9000, 5, 12000, 1], 9, 3),
                                                ([1, 3, 1], [1700, 900, 2], 2, 5)], ids=["most", "many", "few"])
def test_joined_splits(dtype, d, ql, kl, least, behind):
    """Both ways of joining the splits of a row, at each head size, with tokens behind."""
    n = splits(sum(ql) + behind, sum(kl) + behind, len(ql), 3, 1, d, dtype, False)
    assert n >= least and (least > 8 or n <= 8), n
    run_case(dtype, ql, kl, 3, 1, d, back=False, behind=behind, seed=d)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ql,kl,hq,hk,behind,packed", [([900, 0, 1301], [900, 7, 1301], 2, 1, 6, True),
                                                       ([700, 20], [811, 3], 3, 1, 0, True),
                                                       ([1027, 1027], [1027, 1027], 2, 2, 0, False)],
                         ids=["ragged", "groups", "batch"])
def test_split_backward(dtype, d, ql, kl, hq, hk, behind, packed):
    """The rows of a key tile split between workgroups and added: each head size and type,
    several sequences, an empty one, keys before the queries, more queries than keys, tokens
    behind, the batched form."""
    assert splits(sum(ql) + behind, sum(kl) + behind, len(ql), hq, hk, d, dtype, True, packed) > 1
    run_case(dtype, ql, kl, hq, hk, d, packed=packed, behind=behind, seed=d)


def test_arrays_past_31_bits():
    """More than 2^31 elements of q, k, v, o and the gradients; the sequences at both ends are
    what they are by themselves."""
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    H, d, each, n = 64, 128, 64, (1 << 12) + 2
    assert n * each * H * d > 2 ** 31
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v, do = (torch.randn(n * each, H, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    cu = torch.arange(n + 1, device="cuda", dtype=torch.int32) * each
    o, lse = attention_fwd(q, k, v, cu_seqlens=cu)
    g = attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu)
    for i in (0, n // 2, n - 1):
        s = slice(i * each, (i + 1) * each)
        o1, lse1 = attention_fwd(q[s], k[s], v[s], cu_seqlens=offsets([each]))
        g1 = attention_bwd(q[s], k[s], v[s], o1, lse1, do[s], cu_seqlens=offsets([each]))
        assert torch.equal(o[s], o1) and torch.equal(lse[s], lse1), i
        for name in ("dq", "dk", "dv"):
            assert torch.equal(g[name][s], g1[name]), (name, i)


@pytest.mark.parametrize("d", [32, 128])
def test_strides_past_31_bits(d):
    """Tokens as far apart as is allowed: the last ones lie 2^31 elements and more from the first,
    in the inputs, the incoming gradients and the gradients; prompts and a single token."""
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    T, step = 150, 1 << 24
    assert (T - 1) * step > 2 ** 31
    wide = torch.empty(T, step, device="cuda", dtype=torch.bfloat16)
    parts = [rand(i, T, 2, d, dtype="bf16") for i in range(4)]
    at = lambda i: wide[:, i * step // 8:][:, :2 * d].unflatten(1, (2, d))  # noqa: E731
    for i, t in enumerate(parts):
        at(i).copy_(t)
    (q, k, v, do), (wq, wk, wv, wdo, wdq, wdk, wdv) = parts, [at(i) for i in range(7)]
    cu, one = offsets([T]), offsets([1])
    o, lse = attention_fwd(q, k, v, cu_seqlens=cu)
    o2, lse2 = attention_fwd(wq, wk, wv, cu_seqlens=cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    want = attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu)
    got = attention_bwd(wq, wk, wv, o, lse, wdo, cu_seqlens=cu, out=dict(dq=wdq, dk=wdk, dv=wdv))
    for n in ("dq", "dk", "dv"):
        assert torch.equal(want[n], got[n]), n
    o, _ = attention_fwd(q[-1:], k, v, cu_seqlens=one, cu_seqlens_k=cu)
    o2, _ = attention_fwd(wq[-1:], wk, wv, cu_seqlens=one, cu_seqlens_k=cu)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("lens,hq,hk,d,spread", [([1], 2, 2, 64, 1.0), ([2, 1, 9], 4, 1, 128, 1.0), ([64, 3], 2, 2, 32, 2.0),
                                                 ([128], 3, 1, 64, 1.0), ([300], 4, 2, 128, 2.5), ([700, 129], 2, 1, 64, 2.5),
                                                 ([1400], 2, 1, 128, 2.0)])
def test_rounded_results_do_not_reach_the_gradients(lens, hq, hk, d, spread):
    """bf16: D = do . o, which all weights of a row share, is held to fp32 although o is rounded:
    in dk of every length, and in dq of the rows that see 128 keys at most.

    D is formed as D' + sum_j P_ij (do_i . v_j - D'), D' from the rounded o.  With dp_ij the sum of
    absolute values of do_i . v_j and Da that of D: each difference is off by (d + 4) u (dp + Da),
    the weights by ep relatively (and their sum from 1 by ep, which multiplies D'), the sum over
    the keys by (Lk + 16) u."""
    import torch
    from layer_helpers import TINY, U, half
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    total = sum(lens)
    q, do = rand(1, total, hq, d, dtype="bf16", scale=spread), rand(4, total, hq, d, dtype="bf16")
    k, v = rand(2, total, hk, d, dtype="bf16"), rand(3, total, hk, d, dtype="bf16")
    cu = offsets(lens)
    o, lse = attention_fwd(q, k, v, cu_seqlens=cu)
    g = attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu)
    torch.cuda.synchronize()
    Q, K, V, DO, DQ, DK = (f64(t) for t in (q, k, v, do, g["dq"], g["dk"]))
    h, sc = half("bf16"), float(np.float32(d ** -0.5))
    for n, (a, b) in enumerate(L.ranges(lens)):
        T, grp = b - a, hq // hk
        f, r = L.attention(Q[a:b], K[a:b], V[a:b], sc), L.attention_backward(Q[a:b], K[a:b], V[a:b], DO[a:b], sc)
        bq, bk = np.zeros_like(Q[a:b]), np.zeros_like(K[a:b])
        for i in range(hq):
            kv = i // grp
            A = sc * (np.abs(Q[a:b, i]) @ np.abs(K[a:b, kv]).T)
            ep = 2 * ((d + 4) * U * A.max() + U * (A.max() + 4) * 2) + (T + 16) * U
            p, go = f["p"][i], np.abs(DO[a:b, i])
            dp, Da = go @ np.abs(V[a:b, kv]).T, np.sum(go * np.abs(f["o"][:, i]), -1, keepdims=True)
            eD = np.sum(p * ((d + 4) * U + ep + (T + 16) * U) * (dp + Da), -1, keepdims=True) + ep * Da
            eds = p * ((d + 4) * U * (dp + Da) + eD + (ep + 2 * U) * (dp + Da)) + (h + (T * grp + 2) * U) * np.abs(r["ds"][i])
            eds = eds * (1 + h) + TINY
            bq[:, i] = sc * eds @ np.abs(K[a:b, kv])
            bk[:, kv] += sc * eds.T @ np.abs(Q[a:b, i])
        few = min(T, 128)
        check(f"dq[{n}]", DQ[a:a + few], r["dq"][:few], (bq * (1 + h) + h * np.abs(r["dq"]) + TINY)[:few])
        check(f"dk[{n}]", DK[a:b], r["dk"], bk * (1 + h) + h * np.abs(r["dk"]) + TINY)


@pytest.mark.parametrize("lens,hq,hk,d,spread,names", [([2] * 40, 4, 2, 64, 1.0, ("dq", "dk")), ([3, 2, 4] * 9, 2, 2, 128, 1.0, ("dq", "dk")),
                                                       ([128] * 2, 2, 1, 32, 2.0, ("dq", "dk")), ([1500], 4, 1, 128, 2.5, ("dk",))])
def test_gradients_are_as_good_as_their_roundings(lens, hq, hk, d, spread, names):
    """The norm of the error of dq and dk in bf16 is that of the roundings of dS and of the result.

    A rounding of x is off by at most 2^-8 |x| and, over evenly spread remainders, by 2^-8 / sqrt(3)
    |x| in the mean square.  They are independent, so their squares add: over the result's entries,
    and over the terms scale dS_ij k_j (dS_ij q_i) of its sum."""
    import torch
    from recurrent_sequence_models_amd import attention_bwd, attention_fwd
    total, grp, sc = sum(lens), hq // hk, d ** -0.5
    q, do = rand(1, total, hq, d, dtype="bf16", scale=spread), rand(4, total, hq, d, dtype="bf16")
    k, v = rand(2, total, hk, d, dtype="bf16"), rand(3, total, hk, d, dtype="bf16")
    cu = offsets(lens)
    o, lse = attention_fwd(q, k, v, cu_seqlens=cu)
    g = attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu)
    torch.cuda.synchronize()
    Q, K, V, DO = (f64(t) for t in (q, k, v, do))
    err, terms = dict.fromkeys(names, 0.0), dict.fromkeys(names, 0.0)
    for a, b in L.ranges(lens):
        r = L.attention_backward(Q[a:b], K[a:b], V[a:b], DO[a:b], sc)
        for n in names:
            err[n] += np.sum((f64(g[n])[a:b] - r[n]) ** 2)
            terms[n] += np.sum(r[n] ** 2)
        for h in range(hq):
            ds2 = (sc * r["ds"][h]) ** 2
            for n, w in (("dq", ds2 @ np.sum(K[a:b, h // grp] ** 2, -1)), ("dk", ds2.T @ np.sum(Q[a:b, h] ** 2, -1))):
                if n in names:
                    terms[n] += np.sum(w)
    for n in names:
        assert err[n] <= terms[n] * 2.0 ** -16 / 3, (n, np.sqrt(err[n] / terms[n]) / 2.0 ** -8)
