"""CPU pins of the fp64 oracle of a state-space block's operators: torch's own functions and
automatic differentiation in double precision, closed forms and special cases."""

import numpy as np
import pytest
import torch
import torch.nn.functional as TF

from oracle import block as O


def t(a):
    return torch.tensor(a, dtype=torch.float64, requires_grad=True)


def same(a, b, tol=1e-10):
    b = b.detach().numpy() if isinstance(b, torch.Tensor) else b
    np.testing.assert_allclose(a, b, rtol=tol, atol=tol)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_activations(act):
    p = t(np.linspace(-30, 30, 401))
    y = TF.silu(p) if act == "silu" else TF.gelu(p) if act == "gelu" else p * 1
    slope, = torch.autograd.grad(y.sum(), p)
    v, s = O.activation(p.detach().numpy(), act)
    same(v, y)
    same(s, slope)


def test_rms_norm():
    r = np.random.default_rng(0)
    s, w, dy, ds = t(r.normal(size=(5, 12))), t(r.normal(size=12)), r.normal(size=(5, 12)), r.normal(size=(5, 12))
    y = s * w * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6)
    same(O.rms_norm(s.detach().numpy(), w.detach().numpy()), y)
    gs, gw = torch.autograd.grad((torch.tensor(dy) * y).sum() + (torch.tensor(ds) * s).sum(), (s, w))
    dx, dw = O.rms_norm_backward(s.detach().numpy(), w.detach().numpy(), dy, ds)
    same(dx, gs)
    same(dw, gw)
    # a row of equal entries has norm 1 but for eps; scaling the input changes nothing but eps
    same(O.rms_norm(np.full((1, 8), 3.0), np.ones(8), 0.0), np.ones((1, 8)))


@pytest.mark.parametrize("taps,act", [(2, None), (3, "silu"), (4, "silu")])
def test_conv(taps, act):
    r = np.random.default_rng(taps)
    T, D = 9, 5
    x, w, b, s = t(r.normal(size=(T, D))), t(r.normal(size=(D, taps))), t(r.normal(size=D)), t(r.normal(size=(taps - 1, D)))
    dy, df = r.normal(size=(T, D)), r.normal(size=(taps - 1, D))
    ext = torch.cat([s, x])
    y = TF.conv1d(ext.T[None], w[:, None], b, groups=D)[0].T
    y = TF.silu(y) if act else y
    f, final, _ = O.conv(*(a.detach().numpy() for a in (x, w, b, s)), act)
    same(f, y)
    same(final, ext[T:])
    g = torch.autograd.grad((torch.tensor(dy) * y).sum() + (torch.tensor(df) * ext[T:]).sum(), (x, w, b, s))
    o = O.conv_backward(*(a.detach().numpy() for a in (x, w, b, s)), dy, df, act)
    for a, n in zip(g, ("dx", "dw", "db", "dinit")):
        same(o[n], a)


@pytest.mark.parametrize("gate,softplus", [(True, True), (False, True), (True, False)])
def test_ssm(gate, softplus):
    r = np.random.default_rng(7)
    T, D, N = 6, 3, 4
    names = ("x", "dt", "A", "B", "C", "D", "z", "bias", "init")
    v = dict(x=r.normal(size=(T, D)), dt=np.abs(r.normal(size=(T, D))), A=-np.exp(r.normal(size=(D, N))), B=r.normal(size=(T, N)),
             C=r.normal(size=(T, N)), D=r.normal(size=D), z=r.normal(size=(T, D)) if gate else None, bias=r.normal(size=D),
             init=r.normal(size=(D, N)))
    p = {k: None if a is None else t(a) for k, a in v.items()}
    delta = p["dt"] + p["bias"]
    delta = TF.softplus(delta, threshold=1000) if softplus else delta
    h, ys = p["init"], []
    for i in range(T):
        h = torch.exp(delta[i][:, None] * p["A"]) * h + (delta[i] * p["x"][i])[:, None] * p["B"][i]
        ys.append((h * p["C"][i]).sum(-1) + p["D"] * p["x"][i])
    y = torch.stack(ys) * (TF.silu(p["z"]) if gate else 1)
    f = O.ssm(softplus=softplus, **v)
    same(f["y"], y)
    same(f["final"], h)
    dy, df = r.normal(size=(T, D)), r.normal(size=(D, N))
    on = [k for k in names if v[k] is not None]
    g = torch.autograd.grad((torch.tensor(dy) * y).sum() + (torch.tensor(df) * h).sum(), [p[k] for k in on])
    o = O.ssm_backward(dy=dy, d_final=df, softplus=softplus, **v)
    for k, a in zip(on, g):
        same(o["d" + k], a)


def test_ssm_closed_form():
    """Constant decays and inputs: a geometric sum."""
    T, a = 20, 0.7
    x = np.ones((T, 1))
    f = O.ssm(x, np.full((T, 1), 1.0), np.log(np.full((1, 1), a)), np.ones((T, 1)), np.ones((T, 1)), softplus=False)
    same(f["y"][:, 0], (1 - a ** np.arange(1, T + 1)) / (1 - a))


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_linear(act):
    r = np.random.default_rng(2)
    x, w, b, res, dy = t(r.normal(size=(5, 7))), t(r.normal(size=(4, 7))), t(r.normal(size=4)), r.normal(size=(5, 4)), r.normal(size=(5, 4))
    p = TF.linear(x, w, b)
    y = (TF.silu(p) if act == "silu" else TF.gelu(p) if act == "gelu" else p) + torch.tensor(res)
    got, pre = O.linear(*(a.detach().numpy() for a in (x, w, b)), act, res)
    same(got, y)
    g = torch.autograd.grad((torch.tensor(dy) * y).sum(), (x, w, b))
    o = O.linear_backward(x.detach().numpy(), w.detach().numpy(), dy, pre, act)
    for a, n in zip(g, ("dx", "dw", "db")):
        same(o[n], a)
