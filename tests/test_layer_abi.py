"""CPU tests of the layer operators' C ABI: invalid calls are refused on the host before
any HIP call, and workspace sizes follow their formulas.  Pointer arguments are fake
aligned addresses that are never dereferenced, so the refusal tests only run where no GPU
is visible."""

import ctypes

import pytest

from recurrent_sequence_models_amd import falcon as F

P = 0x10000


def _no_gpu():
    try:
        import torch
        return torch.cuda.device_count() == 0
    except Exception:
        return True


cpu_only = pytest.mark.skipif(not _no_gpu(), reason="invalid-call tests run only where no GPU is visible")
ref = ctypes.byref
INVALID, UNSUPPORTED, WORKSPACE = F.ERR_INVALID_ARG, F.ERR_UNSUPPORTED, F.ERR_WORKSPACE


def scan_shape(**kw):
    d = dict(dtype=1, batch=2, seqlen=1000, width=64, input=0)
    d.update(kw)
    return F.ScanShape(*d.values())


BAD_SCAN = [(dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(batch=0), INVALID), (dict(seqlen=0), INVALID),
            (dict(width=0), INVALID), (dict(width=-8), INVALID), (dict(width=12), UNSUPPORTED),
            (dict(input=2), INVALID), (dict(seqlen=2 ** 31 - 10), UNSUPPORTED),
            (dict(batch=2 ** 31 - 1, width=1 << 20), UNSUPPORTED)]


def scan_fwd(s, cu=None, x=P, g=P, init=None, fin=None, h=P, st=None, ws=P, n=1 << 40):
    return F.lib().falcon_scan_fwd(ref(s) if s is not None else None, cu, x, g, init, fin, h, st, ws, n, None)


def scan_bwd(s, cu=None, x=P, g=P, init=None, st=P, dh=P, df=None, dx=P, dg=P, di=None, ws=P, n=1 << 40):
    return F.lib().falcon_scan_bwd(ref(s), cu, x, g, init, st, dh, df, dx, dg, di, ws, n, None)


@cpu_only
def test_scan_refusals():
    L = F.lib()
    for kw, want in BAD_SCAN:
        s = scan_shape(**kw)
        assert scan_fwd(s) == want and scan_bwd(s) == want, kw
        assert L.falcon_scan_workspace(ref(s), 0) == 0
        if "seqlen" not in kw and "batch" not in kw or kw.get("batch") == 0:
            assert L.falcon_scan_step(ref(s), P, P, P, P, None) == want, kw
    s = scan_shape()
    assert scan_fwd(None) == INVALID
    for kw in (dict(x=None), dict(g=None), dict(h=None), dict(x=P + 8), dict(h=P + 2), dict(init=P + 4),
               dict(fin=P + 8), dict(st=P + 4), dict(cu=P + 2), dict(ws=P + 8)):
        assert scan_fwd(s, **kw) == INVALID, kw
    for kw in (dict(x=None), dict(st=None), dict(dh=None), dict(dx=None), dict(dg=P + 8), dict(di=P + 4),
               dict(df=P + 4)):
        assert scan_bwd(s, **kw) == INVALID, kw
    need = L.falcon_scan_workspace(ref(s), 0)
    assert scan_fwd(s, n=need - 1) == WORKSPACE and scan_fwd(s, ws=None) == WORKSPACE
    assert scan_bwd(s, n=need - 1) == WORKSPACE
    for a in ((None, P, P, P), (P, None, P, P), (P, P, None, P), (P, P, P, None), (P + 4, P, P, P)):
        assert L.falcon_scan_step(ref(s), *a, None) == INVALID


def test_scan_workspace():
    """None for one chunk; linear in the columns of 128 bytes; a packed call has one time axis."""
    ws = lambda packed=0, **kw: F.lib().falcon_scan_workspace(ref(scan_shape(**kw)), packed)  # noqa: E731
    assert ws(seqlen=256) == 0 and ws(seqlen=257) > 0
    assert ws(width=128) <= 2 * ws() and ws(width=72) == ws(width=128)
    assert ws(dtype=0, width=32) < ws(dtype=0, width=64)
    assert ws(packed=1, batch=50) == ws(packed=1, batch=1) == ws(batch=1)
    assert ws(batch=4) > ws(batch=2)


def qk_shape(**kw):
    d = dict(dtype=1, tokens=10, heads_q=4, heads_k=2, d=64, rot=32, layout=0, norm=1, eps=1e-6, rot_scale=1.0,
             grad_dtype=1)
    d.update(kw)
    return F.QkShape(*d.values())


def H(p=P, stride=4 * 64):
    return F.Heads(p, stride)


def qk_fwd(s, q=H(), k=H(), wq=P, wk=P, pos=P, freq=P, qo=H(), ko=H()):
    return F.lib().falcon_qk_norm_rope(ref(s) if s is not None else None, q, k, wq, wk, pos, freq, qo, ko, None)


def qk_bwd(s, q=H(), k=H(), wq=P, wk=P, pos=P, freq=P, dqo=H(), dko=H(), dq=H(), dk=H(), dwq=P, dwk=P, ws=P, n=1 << 40):
    return F.lib().falcon_qk_norm_rope_bwd(ref(s), q, k, wq, wk, pos, freq, dqo, dko, dq, dk, dwq, dwk, ws, n, None)


@cpu_only
def test_qk_refusals():
    inf, nan = float("inf"), float("nan")
    for kw, want in [(dict(dtype=3), INVALID), (dict(tokens=0), INVALID), (dict(heads_q=0), INVALID),
                     (dict(heads_k=0), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
                     (dict(rot=24), UNSUPPORTED), (dict(rot=80), INVALID), (dict(rot=-16), INVALID),
                     (dict(layout=2), INVALID), (dict(norm=2), INVALID), (dict(eps=-1.0), INVALID),
                     (dict(eps=nan), INVALID), (dict(rot_scale=inf), INVALID), (dict(grad_dtype=7), INVALID),
                     (dict(heads_q=1 << 21), UNSUPPORTED), (dict(tokens=2 ** 31 - 1), UNSUPPORTED)]:
        s = qk_shape(**kw)
        assert qk_fwd(s) == want and qk_bwd(s) == want, kw
        assert F.lib().falcon_qk_norm_rope_bwd_workspace(ref(s)) == 0
    s = qk_shape()
    assert qk_fwd(None) == INVALID
    for kw in (dict(q=H(None)), dict(k=H(P + 8)), dict(qo=H(None)), dict(ko=H(P, 127)), dict(q=H(P, 255)),
               dict(q=H(P, 257)), dict(q=H(P, -256)), dict(q=H(P, 1 << 62)), dict(pos=None), dict(pos=P + 2),
               dict(freq=None), dict(freq=P + 4), dict(wq=P + 4)):
        assert qk_fwd(s, **kw) == INVALID, kw
        if "qo" not in kw and "ko" not in kw:
            assert qk_bwd(s, **kw) == INVALID, kw
    for kw in (dict(dqo=H(None)), dict(dko=H(P, 100)), dict(dq=H(P + 2)), dict(dwq=P + 2), dict(ws=P + 8)):
        assert qk_bwd(s, **kw) == INVALID, kw
    assert qk_bwd(qk_shape(norm=0), wq=None, wk=None) == INVALID            # a weight gradient without weights
    assert qk_bwd(qk_shape(dtype=0, grad_dtype=1)) == UNSUPPORTED
    need = F.lib().falcon_qk_norm_rope_bwd_workspace(ref(s))
    assert need == 10 * 2 * 64 * 4
    assert qk_bwd(s, n=need - 1) == WORKSPACE and qk_bwd(s, ws=None) == WORKSPACE


def attn_shape(**kw):
    d = dict(dtype=1, batch=2, seqlen_q=100, seqlen_k=100, heads_q=4, heads_k=2, d=64, scale=0.125)
    d.update(kw)
    return F.AttnShape(*d.values())


def attn_fwd(s, cq=None, ck=None, q=H(), k=H(), v=H(), o=P, lse=P, ws=P, n=1 << 40):
    return F.lib().falcon_attn_fwd(ref(s) if s is not None else None, cq, ck, q, k, v, o, lse, ws, n, None)


def attn_bwd(s, cq=None, ck=None, q=H(), k=H(), v=H(), o=P, lse=P, do=H(), dq=H(), dk=H(), dv=H(), ws=P, n=1 << 40):
    return F.lib().falcon_attn_bwd(ref(s), cq, ck, q, k, v, o, lse, do, dq, dk, dv, ws, n, None)


@cpu_only
def test_attention_refusals():
    for kw, want in [(dict(dtype=2), INVALID), (dict(batch=0), INVALID), (dict(seqlen_q=0), INVALID),
                     (dict(seqlen_k=-1), INVALID), (dict(heads_q=3), INVALID), (dict(heads_k=0), INVALID),
                     (dict(d=80), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
                     (dict(scale=-1.0), INVALID), (dict(seqlen_q=2 ** 31 - 1), UNSUPPORTED),
                     (dict(batch=1 << 20, seqlen_k=1 << 20), UNSUPPORTED)]:
        s = attn_shape(**kw)
        assert attn_fwd(s) == want and attn_bwd(s) == want, kw
        assert F.lib().falcon_attn_fwd_workspace(ref(s), 0) == 0 == F.lib().falcon_attn_bwd_workspace(ref(s), 0)
    s = attn_shape()
    assert attn_fwd(None) == INVALID
    for kw in (dict(q=H(None)), dict(k=H(P + 8)), dict(v=H(P, 64)), dict(v=H(P, 129)), dict(o=None), dict(o=P + 8),
               dict(lse=P + 2), dict(cq=P), dict(ck=P), dict(cq=P + 2, ck=P)):
        assert attn_fwd(s, **kw) == INVALID and attn_bwd(s, **kw) == INVALID, kw
    for kw in (dict(lse=None), dict(do=H(None)), dict(dq=H(P + 8)), dict(dk=H(P, 64)), dict(dv=H(None))):
        assert attn_bwd(s, **kw) == INVALID, kw
    assert attn_bwd(s, n=2 * 2 * 100 * 4 * 4 - 1) == WORKSPACE and attn_bwd(s, ws=None) == WORKSPACE
    assert attn_bwd(s, ws=P + 8) == INVALID
    few = attn_shape(seqlen_q=1, seqlen_k=4096)
    need = F.lib().falcon_attn_fwd_workspace(ref(few), 0)
    assert need > 0 and attn_fwd(few, n=need - 1) == WORKSPACE and attn_fwd(few, ws=None) == WORKSPACE
    assert attn_fwd(few, ws=P + 8) == INVALID


def test_attention_workspace():
    """Partial results only where few rows meet many keys; two numbers a row in the backward."""
    L = F.lib()
    assert L.falcon_attn_fwd_workspace(ref(attn_shape()), 0) == 0
    assert L.falcon_attn_fwd_workspace(ref(attn_shape(seqlen_q=1 << 15, seqlen_k=1 << 15)), 0) == 0
    assert L.falcon_attn_fwd_workspace(ref(attn_shape(seqlen_q=2, seqlen_k=1 << 14)), 1) > 0
    assert L.falcon_attn_bwd_workspace(ref(attn_shape()), 0) == 2 * 2 * 100 * 4 * 4
    assert L.falcon_attn_bwd_workspace(ref(attn_shape()), 1) == 2 * 100 * 4 * 4


@cpu_only
def test_sizes_past_a_launch_or_an_index():
    """Sizes whose workgroups, numbers or addresses would pass what a launch or an index holds are
    refused, the largest that fit are not (they get as far as the workspace)."""
    L = F.lib()
    big = 1 << 62
    for kw, packed in ((dict(batch=1 << 23, seqlen=1, width=64), 0), (dict(batch=1 << 22, seqlen=257, width=64), 0),
                       (dict(batch=1, seqlen=1 << 26, width=1 << 12), 1), (dict(batch=(1 << 30) + 1, seqlen=1000), 1)):
        s, cu = scan_shape(**kw), P if packed else None
        assert scan_fwd(s, cu=cu, n=big) == UNSUPPORTED and scan_bwd(s, cu=cu, n=big) == UNSUPPORTED, kw
        assert L.falcon_scan_workspace(ref(s), packed) == 0
    for kw, packed in ((dict(batch=(1 << 22) - 1, seqlen=257, width=64), 0), (dict(batch=1 << 30, seqlen=1000), 1)):
        s, cu = scan_shape(**kw), P if packed else None
        assert scan_fwd(s, cu=cu, n=16) == WORKSPACE and scan_bwd(s, cu=cu, n=16) == WORKSPACE, kw
    assert L.falcon_scan_step(ref(scan_shape(batch=1 << 30, width=1 << 5)), P, P, P, P, None) == UNSUPPORTED
    for kw in (dict(batch=1 << 24, seqlen_q=1, seqlen_k=1, heads_q=8, heads_k=8),
               dict(batch=1 << 12, seqlen_q=1 << 12, seqlen_k=1 << 12, heads_q=256, heads_k=128)):
        s = attn_shape(**kw)
        t = H(P, kw["heads_q"] * 64)
        assert attn_fwd(s, q=t, k=t, v=t, n=big) == UNSUPPORTED, kw
        assert attn_bwd(s, q=t, k=t, v=t, do=t, dq=t, dk=t, dv=t, n=big) == UNSUPPORTED, kw
    assert attn_bwd(attn_shape(batch=1 << 10, seqlen_q=1 << 10, seqlen_k=1), n=16) == WORKSPACE
    for dtype, most in ((1, 1 << 24), (0, 1 << 23)):   # 2^25 bytes between tokens
        s = attn_shape(dtype=dtype)
        for name in ("q", "k", "v"):
            assert attn_fwd(s, **{name: H(P, most + 8)}) == UNSUPPORTED, (dtype, name)
            assert attn_bwd(s, n=16, **{name: H(P, most)}) == WORKSPACE, (dtype, name)
        assert attn_bwd(s, do=H(P, most + 8)) == UNSUPPORTED


def test_sizes_past_32_bits():
    """The binding refuses sizes that the C structs would hold only in part."""
    from recurrent_sequence_models_amd import layer
    for call, sizes in ((layer._scan_plan, (1, 1, 2 ** 32 + 5, 8, False, False)),
                        (layer._qk_plan, (1, 2 ** 32 + 1, 4, 4, 64, 64, 0, 1, 1e-6, 1.0, 1)),
                        (layer._attn_plan, (False, 1, 1, 2 ** 31, 5, 4, 4, 64, 0.125))):
        with pytest.raises(ValueError, match="2\\^31"):
            call(*sizes)
