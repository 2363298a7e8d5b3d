"""CPU tests of the C ABI of a state-space block's operators: invalid calls are refused on the
host before any HIP call, and workspace sizes follow their formulas.  Pointer arguments are fake
aligned addresses that are never dereferenced, so the refusal tests only run where no GPU is
visible."""

import ctypes

import pytest

from recurrent_sequence_models_amd import falcon as F
from test_layer_abi import INVALID, UNSUPPORTED, WORKSPACE, P, cpu_only

Q = 2 * P      # another array

ref = ctypes.byref
BIG = 1 << 62


def shape(kind, defaults):
    def make(**kw):
        d = dict(defaults)
        d.update(kw)
        return kind(*d.values())
    return make


def H(p=Q, stride=64):
    return F.Heads(p, stride)


NONE = F.Heads(None, 0)

norm_shape = shape(F.NormShape, dict(dtype=1, tokens=10, width=64, norm=1, out=1, eps=1e-6))


def norm(s, x=P, res=None, w=P, so=None, y=P, scale=P):
    return F.lib().falcon_rms_norm(ref(s) if s is not None else None, x, res, w, so, y, scale, None)


def norm_bwd(s, st=P, w=P, dy=P, ds=None, dx=P, dw=P, ws=P, n=BIG):
    return F.lib().falcon_rms_norm_bwd(ref(s), st, w, dy, ds, dx, dw, ws, n, None)


@cpu_only
def test_norm_refusals():
    inf, nan = float("inf"), float("nan")
    for kw, want in [(dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(tokens=0), INVALID), (dict(width=0), INVALID),
                     (dict(norm=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=inf), INVALID), (dict(eps=nan), INVALID),
                     (dict(width=12), UNSUPPORTED), (dict(width=32776), UNSUPPORTED), (dict(dtype=0, out=0, width=16392), UNSUPPORTED),
                     (dict(tokens=2 ** 31 - 1), UNSUPPORTED)]:
        s = norm_shape(**kw)
        assert norm(s) == want and norm_bwd(s) == want, kw
        assert F.lib().falcon_rms_norm_bwd_workspace(ref(s)) == 0
    assert norm(None) == INVALID
    assert norm(norm_shape(out=3)) == INVALID and norm(norm_shape(out=0)) == UNSUPPORTED
    assert norm(norm_shape(dtype=0, out=1)) == UNSUPPORTED
    s = norm_shape()
    for kw in (dict(x=None), dict(x=P + 8), dict(res=P + 4), dict(w=P + 4), dict(so=P + 8), dict(y=None), dict(y=P + 2),
               dict(scale=P + 2), dict(res=P, so=2 * P, y=2 * P)):
        assert norm(s, **kw) == INVALID, kw
    assert norm(norm_shape(out=2), y=Q, scale=None) == INVALID
    for kw in (dict(y=P), dict(y=Q, res=Q)):                        # rows of another length
        assert norm(norm_shape(out=2), **kw) == INVALID, kw
    for kw in (dict(st=None), dict(dy=None), dict(dx=None), dict(w=P + 4), dict(ds=P + 8), dict(dw=P + 2), dict(ws=P + 8)):
        assert norm_bwd(s, **kw) == INVALID, kw
    assert norm_bwd(norm_shape(norm=0)) == UNSUPPORTED
    need = F.lib().falcon_rms_norm_bwd_workspace(ref(s))
    assert need == 3 * 64 * 4                                     # 10 rows, 4 a workgroup
    assert norm_bwd(s, n=need - 1) == WORKSPACE and norm_bwd(s, ws=None) == WORKSPACE


conv_shape = shape(F.ConvShape, dict(dtype=1, batch=2, seqlen=100, width=64, taps=4, activation=1))


def conv(s, cu=None, x=H(), w=P, b=P, init=None, fin=None, y=P):
    return F.lib().falcon_conv_fwd(ref(s) if s is not None else None, cu, x, w, b, init, fin, y, None)


def conv_bwd(s, cu=None, x=H(), w=P, b=P, init=None, dy=P, df=None, dx=H(3 * P), dw=P, db=P, di=None, ws=P, n=BIG):
    return F.lib().falcon_conv_bwd(ref(s), cu, x, w, b, init, dy, df, dx, dw, db, di, ws, n, None)


def conv_step(s, x=H(), w=P, b=P, st=P, so=P, y=P):
    return F.lib().falcon_conv_step(ref(s), x, w, b, st, so, y, None)


@cpu_only
def test_conv_refusals():
    L = F.lib()
    for kw, want in [(dict(dtype=2), INVALID), (dict(batch=0), INVALID), (dict(width=0), INVALID), (dict(taps=0), INVALID),
                     (dict(activation=3), INVALID), (dict(activation=-1), INVALID), (dict(activation=2), UNSUPPORTED),
                     (dict(taps=1), UNSUPPORTED), (dict(taps=5), UNSUPPORTED), (dict(width=20), UNSUPPORTED),
                     (dict(width=(1 << 20) + 8), UNSUPPORTED)]:
        s, x = conv_shape(**kw), H(P, 1 << 21)
        assert conv(s, x=x) == want and conv_bwd(s, x=x) == want and conv_step(s, x=x) == want, kw
        assert L.falcon_conv_bwd_workspace(ref(s), 0) == 0
    for kw, want in [(dict(seqlen=0), INVALID), (dict(seqlen=2 ** 31 - 1), UNSUPPORTED), (dict(batch=1 << 16, seqlen=1 << 16), UNSUPPORTED)]:
        s = conv_shape(**kw)
        assert conv(s) == want and conv_bwd(s) == want, kw
    assert conv(None) == INVALID
    s = conv_shape()
    for kw in (dict(x=H(None)), dict(x=H(P + 8)), dict(x=H(P, 56)), dict(x=H(P, 65)), dict(x=H(P, 1 << 62)), dict(w=None), dict(w=P + 2),
               dict(b=P + 2), dict(init=P + 8), dict(cu=P + 2)):
        assert conv(s, **kw) == INVALID and conv_bwd(s, **kw) == INVALID, kw
    for kw in (dict(fin=P + 8), dict(y=None), dict(y=P + 8), dict(init=P, fin=P), dict(y=Q)):
        assert conv(s, **kw) == INVALID, kw
    for kw in (dict(dy=None), dict(df=P + 4), dict(dx=H(None)), dict(dx=H(P, 60)), dict(dw=P + 2), dict(db=P + 2), dict(di=P + 8),
               dict(ws=P + 8), dict(df=P, di=P), dict(dx=H(Q)), dict(dx=H(P))):
        assert conv_bwd(s, **kw) == INVALID, kw
    for kw in (dict(x=H(None)), dict(w=None), dict(st=None), dict(so=None), dict(so=P + 8), dict(y=None)):
        assert conv_step(s, **kw) == INVALID, kw
    need = L.falcon_conv_bwd_workspace(ref(s), 0)
    assert need > 0 and need % (64 * 5 * 4) == 0
    assert conv_bwd(s, n=need - 1) == WORKSPACE and conv_bwd(s, ws=None) == WORKSPACE
    assert L.falcon_conv_bwd_workspace(ref(conv_shape(batch=7, seqlen=200)), 1) == L.falcon_conv_bwd_workspace(ref(s), 0)


ssm_shape = shape(F.SsmShape, dict(dtype=1, batch=2, seqlen=100, width=64, state=16, softplus=1))


def ssm(s, cu=None, x=H(), dt=H(), A=P, B=H(), C=H(), D=P, z=H(), b=P, init=None, fin=None, y=P, cs=None, ws=P, n=BIG):
    return F.lib().falcon_ssm_fwd(ref(s) if s is not None else None, cu, x, dt, A, B, C, D, z, b, init, fin, y, cs, ws, n, None)


def ssm_bwd(s, cu=None, x=H(), dt=H(), A=P, B=H(), C=H(), D=P, z=H(), b=P, cs=P, dy=P, df=None, dx=H(), ddt=H(), dA=P, dB=H(),
            dC=H(), dD=P, dz=H(), db=P, di=None, ws=P, n=BIG):
    return F.lib().falcon_ssm_bwd(ref(s), cu, x, dt, A, B, C, D, z, b, cs, dy, df, dx, ddt, dA, dB, dC, dD, dz, db, di, ws, n, None)


def ssm_step(s, x=H(), dt=H(), A=P, B=H(), C=H(), D=P, z=H(), b=P, st=P, so=P, y=P):
    return F.lib().falcon_ssm_step(ref(s), x, dt, A, B, C, D, z, b, st, so, y, None)


@cpu_only
def test_ssm_refusals():
    L = F.lib()
    far = H(P, 1 << 21)
    for kw, want in [(dict(dtype=2), INVALID), (dict(batch=0), INVALID), (dict(width=0), INVALID), (dict(state=0), INVALID),
                     (dict(softplus=2), INVALID), (dict(state=8), UNSUPPORTED), (dict(state=48), UNSUPPORTED), (dict(width=20), UNSUPPORTED),
                     (dict(width=(1 << 20) + 8), UNSUPPORTED)]:
        s, k = ssm_shape(**kw), dict(x=far, dt=far, z=far)
        assert ssm(s, **k) == want and ssm_bwd(s, **k) == want and ssm_step(s, **k) == want, kw
        assert L.falcon_ssm_chunks(ref(s), 0) == L.falcon_ssm_bwd_workspace(ref(s), 0) == L.falcon_ssm_fwd_workspace(ref(s), 0) == 0
    for kw, want in [(dict(seqlen=0), INVALID), (dict(seqlen=2 ** 31 - 1), UNSUPPORTED), (dict(batch=1 << 16, seqlen=1 << 16), UNSUPPORTED)]:
        s = ssm_shape(**kw)
        assert ssm(s) == want and ssm_bwd(s) == want, kw
    assert ssm(None) == INVALID
    s = ssm_shape()
    ins = (dict(x=H(None)), dict(x=H(P, 56)), dict(dt=H(P + 8)), dict(dt=H(P, 65)), dict(A=None), dict(A=P + 4), dict(B=H(None)),
           dict(B=H(P, 8)), dict(C=H(P, 17)), dict(C=H(None)), dict(D=P + 2), dict(z=H(P + 2)), dict(z=H(P, 32)), dict(b=P + 1))
    for kw in ins:
        assert ssm(s, **kw) == INVALID and ssm_bwd(s, **kw) == INVALID and ssm_step(s, **kw) == INVALID, kw
    for name in ("x", "dt", "B", "C", "z"):                         # 2^24 bytes between tokens
        kw = {name: H(P, (1 << 23) + 8)}
        assert ssm(s, **kw) == UNSUPPORTED and ssm_bwd(s, **kw) == UNSUPPORTED and ssm_step(s, **kw) == UNSUPPORTED, kw
    for kw in (dict(cu=P + 2), dict(init=P + 8), dict(fin=P + 4), dict(y=None), dict(cs=P + 8), dict(init=P, fin=P), dict(y=Q)):
        assert ssm(s, **kw) == INVALID, kw
    for kw in (dict(cu=P + 2), dict(cs=None), dict(dy=None), dict(df=P + 4), dict(dx=H(None)), dict(ddt=H(P, 8)), dict(dA=None), dict(dB=H(None)),
               dict(dC=H(P, 9)), dict(dD=P + 2), dict(dz=H(None)), dict(db=P + 2), dict(di=P + 8), dict(ws=P + 8), dict(df=P, di=P)):
        assert ssm_bwd(s, **kw) == INVALID, kw
    for kw in (dict(st=None), dict(so=P + 4), dict(y=None)):
        assert ssm_step(s, **kw) == INVALID, kw
    need = L.falcon_ssm_bwd_workspace(ref(s), 0)
    assert ssm_bwd(s, n=need - 1) == WORKSPACE and ssm_bwd(s, ws=None) == WORKSPACE
    long = ssm_shape(batch=1, seqlen=4096)
    need = L.falcon_ssm_fwd_workspace(ref(long), 0)
    assert need > 0 and ssm(long, n=need - 1) == WORKSPACE and ssm(long, ws=None) == WORKSPACE and ssm(long, ws=P + 8) == INVALID


def test_ssm_sizes():
    """A kept state every 1024 / N steps of a sequence; workspace only where sequences are cut."""
    L = F.lib()
    for N in (16, 32, 64):
        K = 1024 // N
        assert L.falcon_ssm_chunks(ref(ssm_shape(state=N, seqlen=K + 1)), 0) == 4
        assert L.falcon_ssm_chunks(ref(ssm_shape(state=N, seqlen=10 * K + 1, batch=3)), 1) == 13
    assert L.falcon_ssm_fwd_workspace(ref(ssm_shape()), 0) == 0
    assert L.falcon_ssm_fwd_workspace(ref(ssm_shape(batch=64, seqlen=4096, width=1024)), 0) == 0


linear_shape = shape(F.LinearShape, {"dtype": 1, "tokens": 10, "in": 64, "out": 64, "activation": 1, "out_dtype": 1})


def linear(s, x=H(), w=P, sx=None, sw=None, b=P, r=None, y=P, pre=None, ws=P, n=BIG):
    return F.lib().falcon_linear_fwd(ref(s) if s is not None else None, x, w, sx, sw, b, r, y, pre, ws, n, None)


def linear_bwd(s, x=H(), w=P, pre=P, dy=H(), dx=H(3 * P), dw=Q, db=P, ws=P, n=BIG):
    return F.lib().falcon_linear_bwd(ref(s), x, w, pre, dy, dx, dw, db, ws, n, None)


@cpu_only
def test_linear_refusals():
    L = F.lib()
    far = H(P, 1 << 21)
    for kw, want in [({"dtype": 3}, INVALID), ({"out_dtype": 2}, INVALID), ({"tokens": 0}, INVALID), ({"in": 0}, INVALID), ({"out": -8}, INVALID),
                     ({"activation": 3}, INVALID), ({"out_dtype": 0}, UNSUPPORTED), ({"in": 24}, UNSUPPORTED), ({"out": 12}, UNSUPPORTED),
                     ({"in": (1 << 20) + 16}, UNSUPPORTED), ({"out": (1 << 20) + 8}, UNSUPPORTED), ({"tokens": 2 ** 31 - 1}, UNSUPPORTED),
                     ({"tokens": 1 << 30, "out": 1 << 20}, UNSUPPORTED)]:
        s = linear_shape(**kw)
        assert linear(s, x=far) == want and linear_bwd(s, x=far, dy=far, dx=far) == want, kw
        assert L.falcon_linear_fwd_workspace(ref(s)) == L.falcon_linear_bwd_workspace(ref(s)) == 0
    assert linear(None) == INVALID
    s = linear_shape()
    for kw in (dict(x=H(None)), dict(x=H(P, 56)), dict(x=H(P, 65)), dict(w=None), dict(w=P + 8), dict(sx=P, sw=P), dict(sx=P), dict(b=P + 2),
               dict(r=P + 8), dict(y=None), dict(y=P + 8), dict(pre=P + 4), dict(pre=P),
               dict(y=Q), dict(r=Q, pre=Q)):
        assert linear(s, **kw) == INVALID, kw
    assert linear(s, x=H(P, (1 << 22) + 8)) == UNSUPPORTED          # 2^23 bytes between tokens
    q = linear_shape(dtype=2)
    for kw in (dict(), dict(sx=P), dict(sw=P), dict(sx=P + 2, sw=P), dict(sx=P, sw=P, x=H(P, 72))):
        assert linear(q, **kw) == INVALID, kw
    assert linear_bwd(q) == UNSUPPORTED and L.falcon_linear_bwd_workspace(ref(q)) == 0
    for kw in (dict(x=H(None)), dict(w=None), dict(pre=None), dict(pre=P + 8), dict(dy=H(None)), dict(dy=H(P, 8)), dict(dx=H(P, 8)),
               dict(dw=P + 8), dict(db=P + 2), dict(ws=P + 8), dict(dx=H(Q)), dict(x=H(3 * P)), dict(dw=P)):
        assert linear_bwd(s, **kw) == INVALID, kw
    assert linear_bwd(s, dy=H(P, (1 << 22) + 8)) == UNSUPPORTED
    need = L.falcon_linear_bwd_workspace(ref(s))
    assert need > 0 and linear_bwd(s, n=need - 1) == WORKSPACE and linear_bwd(s, ws=None) == WORKSPACE
    mid = linear_shape(**{"tokens": 128, "in": 2048})
    need = L.falcon_linear_fwd_workspace(ref(mid))
    assert need > 0 and linear(mid, x=H(Q, 2048), n=need - 1) == WORKSPACE and linear(mid, x=H(Q, 2048), ws=None) == WORKSPACE


def test_linear_workspace():
    """No partial sums for few tokens on short rows, nor where the tiles fill the chip."""
    L = F.lib()
    size = lambda **kw: L.falcon_linear_fwd_workspace(ref(linear_shape(**kw)))  # noqa: E731
    assert size(**{"tokens": 16, "in": 2048, "out": 4096}) == 0
    assert size(**{"tokens": 65, "in": 2048, "out": 2048}) > 0
    assert size(**{"tokens": 16384, "in": 2048, "out": 2048}) == 0


def test_sizes_past_32_bits():
    """The binding refuses sizes that the C structs would hold only in part."""
    from recurrent_sequence_models_amd import block
    for call, sizes in ((block._norm_plan, (1, 2 ** 32 + 1, 64, 1, 1, 1e-6)), (block._conv_plan, (1, 1, 2 ** 32 + 5, 8, 4, 1, False)),
                        (block._ssm_plan, (1, 2 ** 31, 1, 8, 16, 1, False)), (block._linear_plan, (1, 2 ** 32 + 64, 64, 64, 0, 1))):
        with pytest.raises(ValueError, match="2\\^31"):
            call(*sizes)


# ---- The same array as input and output, where others read it late --------------------------------

def at(k):
    """The k-th of arrays that are not the same."""
    return (k + 1) * P


CONV = dict(x=H(at(0)), w=at(1), b=at(2), init=at(3), dy=at(4), df=at(5), dx=H(at(6)), dw=at(7), db=at(8), di=at(9), ws=at(10))


@cpu_only
def test_conv_bwd_initial_state_and_its_gradient():
    """The run that owns a sequence's first token writes d_init, while runs behind it may read init still."""
    for cu in (None, at(11)):
        assert conv_bwd(conv_shape(), cu=cu, **{**CONV, "di": CONV["init"]}) == INVALID


LINEAR = dict(x=H(at(0)), w=at(1), b=at(2), r=at(3), y=at(4), pre=at(5), ws=at(6))


@cpu_only
@pytest.mark.parametrize("out,ins", [("y", "w sx sw b"), ("pre", "x w sx sw b")])
def test_linear_outputs_over_operands(out, ins):
    """Workgroups store their tiles while others copy operands still, and rows while others read scales and the bias."""
    bits, more = linear_shape(dtype=2, out_dtype=0), dict(sx=at(7), sw=at(8))
    for name in ins.split():
        for s, call in ((linear_shape(), LINEAR), (linear_shape(dtype=0, out_dtype=0), LINEAR), (bits, {**LINEAR, **more})):
            if name in call:
                p = call[name]
                assert linear(s, **{**call, out: p.data if name == "x" else p}) == INVALID, name
    assert linear(linear_shape(), **{**LINEAR, "pre": LINEAR["y"]}) == INVALID


BACK = dict(x=H(at(0)), w=at(1), pre=at(2), dy=H(at(3)), dx=H(at(4)), dw=at(5), db=at(6), ws=at(7))


@cpu_only
@pytest.mark.parametrize("out,ins", [("dx", "w"), ("dw", "x dy"), ("db", "x w dy")])
def test_linear_bwd_outputs_over_operands(out, ins):
    """The products run after the bias's gradient, dx before dweight, and copy operands while tiles are stored."""
    as_out = H if out == "dx" else (lambda p: p)
    for name in ins.split():
        p = BACK[name]
        for act in (0, 1):
            assert linear_bwd(linear_shape(activation=act), **{**BACK, out: as_out(getattr(p, "data", p))}) == INVALID, name
    for other in {"dx", "dw", "db"} - {out}:
        p = BACK[other]
        assert linear_bwd(linear_shape(), **{**BACK, out: as_out(getattr(p, "data", p))}) == INVALID, other


CSTEP = dict(x=H(at(0)), w=at(1), b=at(2), st=at(3), so=at(4), y=at(5))
SSTEP = dict(x=H(at(0)), dt=H(at(1)), A=at(2), B=H(at(3)), C=H(at(4)), D=at(5), z=H(at(6)), b=at(7), st=at(8), so=at(9), y=at(10))


def refused(call, s, args, out, ins, code=INVALID):
    for name in ins.split():
        p = args[name]
        assert call(s, **{**args, out: getattr(p, "data", p)}) == code, (out, name)


@cpu_only
def test_single_tokens_over_what_others_read():
    """Filters, and B and C, are read for every sequence or channel; rows of another stride are other tokens' too."""
    s, t = conv_shape(), ssm_shape()
    refused(conv_step, s, CSTEP, "y", "w b st so")
    refused(conv_step, s, CSTEP, "so", "x w b")
    refused(ssm_step, t, SSTEP, "y", "A B C D b st so")
    refused(ssm_step, t, SSTEP, "so", "x dt A B C D z b")
    refused(conv_step, s, {**CSTEP, "x": H(at(0), 128)}, "y", "x")
    for name in ("x", "dt", "z"):
        refused(ssm_step, t, {**SSTEP, name: H(at(0), 128)}, "y", name)


SCAN = dict(x=H(at(0)), dt=H(at(1)), A=at(2), B=H(at(3)), C=H(at(4)), D=at(5), z=H(at(6)), b=at(7), init=at(8), fin=at(9), y=at(10),
            cs=at(11), ws=at(12))
SBACK = {**{k: SCAN[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "b")}, "cs": at(8), "dy": at(9), "df": at(10), "dx": H(at(11)),
         "ddt": H(at(12)), "dA": at(13), "dB": H(at(14)), "dC": H(at(15)), "dD": at(16), "dz": H(at(17)), "db": at(18), "di": at(19),
         "ws": at(20)}


@cpu_only
def test_scan_outputs_over_what_others_read():
    """Workgroups of other channels and segments read B, C, the parameters and states late."""
    s = ssm_shape()
    refused(ssm, s, SCAN, "y", "A B C D b init fin cs")
    refused(ssm, s, SCAN, "fin", "x dt A B C D z b init cs")
    refused(ssm, s, SCAN, "cs", "x dt A B C D z b init")
    for name in ("x", "dt", "z"):
        refused(ssm, s, {**SCAN, name: H(at(0), 128)}, "y", name)


@cpu_only
def test_scan_gradients_over_what_others_read():
    s = ssm_shape()
    rows = ("dx", "ddt", "dz", "dB", "dC")
    for out in rows + ("dA", "dD", "db", "di"):
        others = [k for k in rows + ("dA", "dD", "db", "di") if k != out]
        late = ["A", "B", "C", "D", "b", "cs", "df"] * (out in ("dx", "ddt", "dz")) + ["x", "dt", "z", "A", "B", "C", "D", "b", "cs", "dy", "df"] * (out == "di")
        for name in others + late:
            p = SBACK[name]
            p = getattr(p, "data", p)
            assert ssm_bwd(s, **{**SBACK, out: H(p) if out in rows else p}) == INVALID, (out, name)
    for out in ("dx", "ddt", "dz"):
        for name in ("x", "dt", "z"):
            assert ssm_bwd(s, **{**SBACK, name: H(at(0), 128), out: H(at(0))}) == INVALID, (out, name)
            assert ssm_bwd(s, **{**SBACK, out: H(SBACK[name].data, 128)}) == INVALID, (out, name)
        assert ssm_bwd(s, **{**SBACK, out: H(SBACK["dy"], 128)}) == INVALID, out


@cpu_only
def test_conv_outputs_over_what_others_read():
    """Filters are read for every run; the states before and behind a sequence by its first and its last ones."""
    s = conv_shape()
    fwd = {**{k: CONV[k] for k in ("x", "w", "b", "init")}, "fin": at(4), "y": at(5)}
    refused(conv, s, fwd, "y", "x w b init fin")
    refused(conv, s, fwd, "fin", "x w b init")
    for out, ins in (("dx", "x w b init dy df dw db di"), ("di", "x w b init dy df dx dw db"), ("dw", "db")):
        for name in ins.split():
            p = getattr(CONV[name], "data", CONV[name])
            assert conv_bwd(s, **{**CONV, out: H(p) if out == "dx" else p}) == INVALID, (out, name)


@cpu_only
def test_norm_outputs_over_what_others_read():
    """The weight is read for every row, and a row's scale may stand where another row's entries are."""
    args = dict(x=at(0), res=at(1), w=at(2), so=at(3), y=at(4), scale=at(5))
    for s in (norm_shape(), norm_shape(out=2)):
        refused(norm, s, args, "y", "w so")
        refused(norm, s, args, "so", "w")
    refused(norm, norm_shape(out=2), args, "scale", "x res w so y")
    back = dict(st=at(0), w=at(1), dy=at(2), ds=at(3), dx=at(4), dw=at(5), ws=at(6))
    refused(norm_bwd, norm_shape(), back, "dx", "w dw")
