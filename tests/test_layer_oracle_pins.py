"""CPU pins of the layer operators' oracles (oracle/layer_oracle.py): closed forms,
special cases and central differences; and of rope_frequencies."""

import math

import numpy as np
import pytest

from oracle import layer as L


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def differences(f, arrays, directions, h=1e-6):
    """d/dt f(arrays + t directions) at 0, by central differences."""
    up = f(*[a + h * d for a, d in zip(arrays, directions)])
    down = f(*[a - h * d for a, d in zip(arrays, directions)])
    return (up - down) / (2 * h)


# ---- Gated linear recurrence --------------------------------------------------------

@pytest.mark.parametrize("mix", [False, True])
def test_scan_is_the_weighted_sum_of_its_inputs(mix):
    """h_t = sum_s (prod_{s<r<=t} lam_r) u_s + (prod_{r<=t} lam_r) h_0, written out."""
    r = rng(1)
    T, D = 9, 5
    x, g, h0 = r.normal(size=(T, D)), -r.random((T, D)), r.normal(size=D)
    lam = np.exp(g)
    u = (1 - lam) * x if mix else x
    h, fin = L.gated_scan(x, g, h0, mix)
    for t in range(T):
        want = np.prod(lam[:t + 1], 0) * h0 + sum(np.prod(lam[s + 1:t + 1], 0) * u[s] for s in range(t + 1))
        assert np.allclose(h[t], want, atol=1e-13)
    assert np.array_equal(fin, h[-1])


def test_scan_closed_forms():
    """Decay 1 adds up; decay 0 (log -inf) keeps the last input; a constant decay under
    mix leaves a constant input's state where it is."""
    x = rng(2).normal(size=(7, 3))
    assert np.allclose(L.gated_scan(x, np.zeros_like(x))[0], np.cumsum(x, 0))
    assert np.allclose(L.gated_scan(x, np.full_like(x, -np.inf))[0], x)
    c = np.full((6, 2), 1.7)
    assert np.allclose(L.gated_scan(c, np.full_like(c, -0.3), np.full(2, 1.7), mix=True)[0], 1.7)


@pytest.mark.parametrize("mix", [False, True])
def test_scan_gradients_are_differences(mix):
    r = rng(3)
    T, D = 6, 4
    x, g, h0 = r.normal(size=(T, D)), -0.05 - r.random((T, D)), r.normal(size=D)
    dh, df = r.normal(size=(T, D)), r.normal(size=D)
    gr = L.gated_scan_backward(x, g, dh, df, h0, mix)

    def f(x, g, h0):
        h, fin = L.gated_scan(x, g, h0, mix)
        return np.sum(h * dh) + np.sum(fin * df)

    for _ in range(4):
        dirs = [r.normal(size=a.shape) for a in (x, g, h0)]
        want = differences(f, (x, g, h0), dirs)
        got = sum(np.sum(gr[n] * d) for n, d in zip(("dx", "dg", "d_init"), dirs))
        assert got == pytest.approx(want, rel=1e-6, abs=1e-7)


# ---- Norm and rotary positions ---------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_turn(layout):
    """The pairs are complex numbers times e^{i pos f}; norms and the scalar product of
    two rows a fixed distance apart do not depend on where they stand."""
    r = rng(4)
    z = r.normal(size=(3, 2, 12))
    f = 100.0 ** (-np.arange(4) / 4)
    pos = np.array([0, 5, 17])
    y = L.rotate(z, pos, f, layout)
    a, b = (np.arange(4), np.arange(4) + 4) if layout == "half" else (np.arange(4) * 2, np.arange(4) * 2 + 1)
    for n in range(3):
        want = (z[n][:, a] + 1j * z[n][:, b]) * np.exp(1j * pos[n] * f)
        assert np.allclose(y[n][:, a] + 1j * y[n][:, b], want)
    assert np.array_equal(y[0], z[0]) and np.array_equal(y[..., 8:], z[..., 8:])
    q, k = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))
    dots = [np.sum(L.rotate(q, [p + 9], f, layout) * L.rotate(k, [p], f, layout)) for p in (0, 3, 1000)]
    assert np.allclose(dots, dots[0])


def test_norm_closed_form():
    x = np.full((1, 1, 16), 3.0)
    y = L.norm_rope(x, np.arange(16.0), [0], np.ones(4), eps=0.0)
    assert np.allclose(y[0, 0], np.arange(16.0))


@pytest.mark.parametrize("layout,norm", [("half", True), ("interleaved", True), ("half", False)])
def test_norm_rope_gradients_are_differences(layout, norm):
    r = rng(5)
    x, w, dy = r.normal(size=(3, 2, 16)), 1 + 0.3 * r.normal(size=16), r.normal(size=(3, 2, 16))
    f, pos = 50.0 ** (-np.arange(5) / 5), [3, 1, 40]
    kw = dict(norm=norm, eps=1e-3, layout=layout, scale=1.2)
    dx, dw = L.norm_rope_backward(x, w, pos, f, dy, **kw)
    for _ in range(3):
        d1, d2 = r.normal(size=x.shape), r.normal(size=16)
        want = differences(lambda x, w: np.sum(L.norm_rope(x, w, pos, f, **kw) * dy), (x, w), (d1, d2))
        got = np.sum(dx * d1) + (np.sum(dw * d2) if norm else 0.0)
        assert got == pytest.approx(want, rel=1e-6, abs=1e-7)


def test_rope_frequencies():
    """The plain frequencies, and what each scaling does to the fastest and slowest pair."""
    from recurrent_sequence_models_amd import rope_frequencies as rf
    R, s = 64, 8.0
    f, one = rf(R, 10000.0)
    assert one == 1.0 and f.dtype.is_floating_point and f.numel() == R // 2
    assert np.allclose(f.numpy(), [10000.0 ** (-2 * j / R) for j in range(R // 2)], rtol=1e-15)
    assert np.allclose(rf(R, scaling="linear", factor=s)[0].numpy(), f.numpy() / s)
    n = rf(R, scaling="ntk", factor=s)[0]
    assert n[0] == f[0] and n[-1].item() == pytest.approx(f[-1].item() / s)
    p, scale = rf(R, scaling="parts", factor=s, original_length=4096)
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert np.allclose(p.numpy()[turns > 40], f.numpy()[turns > 40])        # beta_fast is 32: a ramp's width beyond
    assert np.allclose(p.numpy()[turns < 0.7], f.numpy()[turns < 0.7] / s)
    assert np.all(p.numpy() <= f.numpy()) and np.all(p.numpy() >= f.numpy() / s)
    assert scale == pytest.approx(0.1 * math.log(s) + 1)
    same, scale = rf(R, scaling="parts", factor=1.0, original_length=4096)
    assert np.allclose(same.numpy(), f.numpy()) and scale == 1.0
    for bad in (dict(rot=7), dict(rot=0), dict(rot=R, scaling="other"), dict(rot=R, scaling="parts"),
                dict(rot=2, scaling="ntk"), dict(rot=R, factor=0.0), dict(rot=R, base=-1.0)):
        with pytest.raises(ValueError):
            rf(**bad)


@pytest.mark.parametrize("base", [1e4, 5e5])
@pytest.mark.parametrize("rot,factor", [(128, 4.0), (64, 8.0), (16, 2.0)])
@pytest.mark.parametrize("length", [100, 4096, 65536, 131072, 10 ** 7, 10 ** 12])
def test_rope_frequencies_by_parts_pair_for_pair(base, rot, factor, length):
    """Every pair from how often it turns: the ramp begins at the last pair that turns at least
    beta_fast = 32 times and ends at the first that turns at most beta_slow = 1 times, counted on
    past the last pair (up to rot - 1) where the slowest still turns more often."""
    from recurrent_sequence_models_amd import rope_frequencies as rf
    f = rf(rot, base)[0].numpy()
    turns = length / (2 * math.pi) * base ** (-2.0 * np.arange(-1, 4 * rot) / rot)
    low = max(int(np.sum(turns >= 32.0)) - 2, 0)
    high = min(int(np.sum(turns > 1.0)) - 1, rot - 1)
    want = [f[j] if j <= low else f[j] / factor if j >= high else
            f[j] * (1 + (1 / factor - 1) * (j - low) / (high - low)) for j in range(rot // 2)]
    got, scale = rf(rot, base, scaling="parts", factor=factor, original_length=length)
    assert np.allclose(got.numpy(), want, rtol=1e-12, atol=0)
    assert scale == pytest.approx(0.1 * math.log(factor) + 1)


@pytest.mark.parametrize("bad", [dict(base=0.5), dict(base=1.0), dict(beta_fast=1.0, beta_slow=32.0), dict(beta_slow=0.0),
                                 dict(original_length=-5), dict(original_length=0), dict(factor=float("inf")),
                                 dict(factor=float("nan")), dict(base=float("inf"))])
def test_rope_frequencies_by_parts_refusals(bad):
    """What has no ramp from the pairs that turn often to those that turn rarely is refused."""
    from recurrent_sequence_models_amd import rope_frequencies as rf
    with pytest.raises(ValueError, match="parts|finite"):
        rf(64, **{**dict(scaling="parts", factor=4.0, original_length=4096), **bad})


# ---- Attention ----------------------------------------------------------------------------

def test_attention_closed_forms():
    """Equal scores give the mean of the values seen; one far larger score gives its
    value; a query before the first key sees nothing."""
    r = rng(6)
    v = r.normal(size=(5, 1, 4))
    f = L.attention(np.zeros((5, 2, 4)), r.normal(size=(5, 1, 4)), v)
    for i in range(5):
        assert np.allclose(f["o"][i, 0], v[:i + 1, 0].mean(0)) and f["lse"][i, 1] == pytest.approx(math.log(i + 1))
    k = np.zeros((4, 1, 4))
    k[1] = 100.0
    f = L.attention(np.ones((1, 1, 4)), k, v[:4])
    assert np.allclose(f["o"][0, 0], v[1, 0])
    f = L.attention(np.ones((3, 1, 4)), k[:1], v[:1])          # three queries, one key
    assert np.all(f["o"][:2] == 0) and np.all(np.isneginf(f["lse"][:2])) and np.allclose(f["o"][2], v[0])


def test_attention_heads_share_keys():
    """Grouped heads are ungrouped heads with repeated keys; their dk, dv add up."""
    r = rng(7)
    q, do = r.normal(size=(2, 3, 6, 4))
    k, v = r.normal(size=(2, 5, 2, 4))
    rep = lambda a: np.repeat(a, 3, axis=1)  # noqa: E731
    assert np.allclose(L.attention(q, k, v)["o"], L.attention(q, rep(k), rep(v))["o"])
    a, b = L.attention_backward(q, k, v, do), L.attention_backward(q, rep(k), rep(v), do)
    assert np.allclose(a["dq"], b["dq"])
    for n in ("dk", "dv"):
        assert np.allclose(a[n], b[n].reshape(5, 2, 3, 4).sum(2))


def test_attention_gradients_are_differences():
    r = rng(8)
    q, do = r.normal(size=(2, 4, 4, 8))
    k, v = r.normal(size=(2, 3, 2, 8))            # the first query sees nothing
    g = L.attention_backward(q, k, v, do, 0.7)
    for _ in range(4):
        dirs = [r.normal(size=a.shape) for a in (q, k, v)]
        want = differences(lambda q, k, v: np.sum(L.attention(q, k, v, 0.7)["o"] * do), (q, k, v), dirs)
        got = sum(np.sum(g[n] * d) for n, d in zip(("dq", "dk", "dv"), dirs))
        assert got == pytest.approx(want, rel=1e-6, abs=1e-7)
    assert np.all(g["dq"][0] == 0)
