"""GPU tests of the norm of the residual stream, its output in 8 bits and its backward pass,
elementwise against the fp64 definition.

Bounds, with u = 2^-24: a sum over a row of D entries is formed as D / 64 sequential sums and a
tree, so it is off by (D / 64 + 16) u of the sum of absolute values; everything else is a few
roundings; results are rounded once to their type (half)."""

import numpy as np
import pytest

from block_helpers import TINY, U, check, f64, half, rand, same_in_graph
from oracle import block as O

pytestmark = pytest.mark.gpu

# one wave a row with each count of 16-byte pieces, the borders between them, and a workgroup a row
SIZES = [(1, 8), (3, 72), (5, 768), (130, 1024), (67, 2048), (9, 2056), (33, 4096), (4, 4104), (2, 16384), (5003, 64)]


def row_err(D):
    return (D / 64 + 20) * U


def norm_bound(s, w, dtype, eps=1e-6):
    return (row_err(s.shape[-1]) + half(dtype)) * np.abs(O.rms_norm(s, w, eps)) + TINY


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,D", SIZES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(dtype, tokens, D, residual):
    import torch
    import recurrent_sequence_models_amd as rsm
    x, res, w = rand(1, tokens, D, dtype=dtype), rand(2, tokens, D, dtype=dtype, scale=3.0), 1 + 0.3 * rand(3, D)
    y, s, scale = rsm.rms_norm(x, w, residual=res if residual else None)
    assert scale is None
    if residual:
        assert torch.equal(s, (x.float() + res.float()).to(x.dtype))
    else:
        assert s is x
    check("y", f64(y), O.rms_norm(f64(s), f64(w)), norm_bound(f64(s), f64(w), dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,D", SIZES)
def test_eight_bits(dtype, tokens, D):
    """q scale is the norm within half a step of e4m3 (2^-4 of a normal number, 2^-10 below them)."""
    import torch
    import recurrent_sequence_models_amd as rsm
    x, res, w = rand(1, tokens, D, dtype=dtype), rand(2, tokens, D, dtype=dtype), 1 + 0.3 * rand(3, D)
    q, s, scale = rsm.rms_norm(x, w, residual=res, quantize=True)
    assert q.dtype is torch.float8_e4m3fn and scale.shape == (tokens,)
    want = O.rms_norm(f64(s), f64(w))
    top = np.abs(want).max(-1)
    check("scale", f64(scale), top / 448, (row_err(D) + 2 * U) * top / 448)
    unit = want / f64(scale)[:, None]
    check("q", f64(q.float()), unit, (2.0 ** -4 + 2 * row_err(D)) * np.abs(unit) + 2.0 ** -10 * (1 + 1e-5))
    assert np.all(np.abs(f64(q.float())).max(-1) == 448)
    q, scale = rsm.quantize_rows(x)
    X = f64(x)
    top = np.abs(X).max(-1) / 448
    check("scale of rows", f64(scale), top, U * top)          # one rounding, of the division
    unit = X / f64(scale)[:, None]
    check("rows", f64(q.float()), unit, (2.0 ** -4 + 4 * U) * np.abs(unit) + 2.0 ** -10)


def test_eight_bits_round_as_the_type_does():
    """Numbers of the 8-bit grid pass as they are, and values between two round to nearest even."""
    import torch
    import recurrent_sequence_models_amd as rsm
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()     # 0 .. 448
    mid = (grid[1:] + grid[:-1]) / 2
    v = torch.cat([grid, -grid, mid, -mid])
    v = torch.cat([v, torch.zeros(-v.numel() % 8)]).cuda()[None]
    q, scale = rsm.quantize_rows(v)
    assert scale.item() == 1.0 and torch.equal(q.float(), v.to(torch.float8_e4m3fn).float())


def test_rows_of_zeros_and_of_no_numbers():
    import torch
    import recurrent_sequence_models_amd as rsm
    for dtype in ("bf16", "fp32"):
        x = rand(1, 6, 200, dtype=dtype)
        x[1], x[3, 7], x[5, 100] = 0, float("nan"), float("inf")
        w = torch.ones(200, device="cuda")
        y, _, _ = rsm.rms_norm(x, w)
        q, _, scale = rsm.rms_norm(x, w, quantize=True)
        p, raw = rsm.quantize_rows(x)
        assert torch.all(y[1] == 0) and torch.all(q[1].float() == 0) and torch.all(p[1].float() == 0)
        assert torch.isfinite(scale[[0, 1, 2, 4]]).all() and scale[1] > 0
        assert torch.isnan(y[3]).all() and torch.isnan(scale[3]) and torch.isnan(raw[3])
        assert torch.isnan(y[5, 100]) and torch.isnan(scale[5])                # inf / inf
        assert torch.isinf(raw[5]) and torch.isnan(p[5, 100].float()) and torch.all(p[5, :100].float() == 0)
        for row in (0, 2, 4):
            alone, _, _ = rsm.rms_norm(x[row:row + 1].clone(), w)
            assert torch.equal(alone[0], y[row]) and torch.isfinite(y[row]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,D", SIZES)
@pytest.mark.parametrize("more", [True, False])
def test_backward(dtype, tokens, D, more):
    """more: a gradient of the stream, and a weight."""
    import recurrent_sequence_models_amd as rsm
    s, dy, ds, w = rand(1, tokens, D, dtype=dtype), rand(2, tokens, D, dtype=dtype), rand(3, tokens, D, dtype=dtype), 1 + 0.3 * rand(4, D)
    g = rsm.rms_norm_bwd(s, w if more else None, dy, d_stream=ds if more else None)
    S, G, W = f64(s), f64(dy), f64(w) if more else np.ones(D)
    dx, dw = O.rms_norm_backward(S, W, G, f64(ds) if more else 0.0)
    r = 1 / np.sqrt((S * S).mean(-1, keepdims=True) + 1e-6)
    v, e = np.abs(S * r), row_err(D)
    # r is off by e; the mean by 3 e of that of absolute values; then a few roundings
    bound = r * (2 * e * np.abs(W * G) + 5 * e * v * np.abs(W * G * S * r).mean(-1, keepdims=True)) + 4 * U * np.abs(dx)
    check("dx", f64(g["dx"]), dx, bound + half(dtype) * np.abs(dx) + 4 * U * (np.abs(f64(ds)) if more else 0) + TINY)
    if more:
        check("dw", f64(g["dweight"]), dw, (tokens / 16 + 100 + D / 64 + 24) * U * np.abs(G * v).sum(0) + TINY)
    else:
        assert g["dweight"] is None


def test_gradients_are_those_of_differences():
    """The definition's gradients against central differences of its values, in 64 bits."""
    r = np.random.default_rng(5)
    s, w, dy = r.normal(size=(3, 24)), 1 + 0.3 * r.normal(size=24), r.normal(size=(3, 24))
    dx, dw = O.rms_norm_backward(s, w, dy)
    for a, grad in ((s, dx), (w, dw)):
        d = r.normal(size=a.shape)
        h = 1e-6
        f = lambda t: (dy * (O.rms_norm(s + t * d, w) if a is s else O.rms_norm(s, w + t * d))).sum()  # noqa: E731
        assert abs((f(h) - f(-h)) / (2 * h) - (grad * d).sum()) < 1e-7


def test_in_place_strays_and_streams():
    """Outputs over inputs, rows behind the last as they were, another stream, and a captured pass."""
    import torch
    import recurrent_sequence_models_amd as rsm
    x, res, w = rand(1, 37, 768, dtype="bf16"), rand(2, 37, 768, dtype="bf16"), 1 + 0.3 * rand(3, 768)
    y, s, _ = rsm.rms_norm(x, w, residual=res)
    a, b = x.clone(), res.clone()
    y2, s2, _ = rsm.rms_norm(a, w, residual=b, out=a, stream_out=b)
    assert y2 is a and s2 is b and torch.equal(a, y) and torch.equal(b, s)
    dy, ds = rand(4, 37, 768, dtype="bf16"), rand(5, 37, 768, dtype="bf16")
    g = rsm.rms_norm_bwd(s, w, dy, d_stream=ds)
    c = ds.clone()
    g2 = rsm.rms_norm_bwd(s, w, dy, d_stream=c, out=c)
    assert torch.equal(g["dx"], c) and torch.equal(g["dweight"], g2["dweight"])
    room = torch.full((40, 768), 7.0, dtype=torch.bfloat16, device="cuda")
    rsm.rms_norm(x, w, residual=res, out=room[:37])
    assert torch.equal(room[:37], y) and torch.all(room[37:] == 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3, _, _ = rsm.rms_norm(x, w, residual=res, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y3, y)

    def call():
        y, s, _ = rsm.rms_norm(x, w, residual=res)
        q, _, scale = rsm.rms_norm(x, w, residual=res, quantize=True)
        g = rsm.rms_norm_bwd(s, w, dy, d_stream=ds)
        return [y, s, q.view(torch.uint8), scale, g["dx"], g["dweight"]]
    same_in_graph(call)


def test_past_32_bits():
    """Rows behind 2^31 entries."""
    import torch
    import recurrent_sequence_models_amd as rsm
    D, tokens = 16384, (1 << 17) + 9
    x = torch.zeros(tokens, D, dtype=torch.bfloat16, device="cuda")
    x[-5:] = rand(1, 5, D, dtype="bf16")
    w = 1 + 0.3 * rand(2, D)
    y, _, _ = rsm.rms_norm(x, w)
    alone, _, _ = rsm.rms_norm(x[-5:].clone(), w)
    assert torch.equal(y[-5:], alone) and torch.all(y[:-5].abs().amax(-1) == 0)
    g = rsm.rms_norm_bwd(x, w, y, out=y)
    h = rsm.rms_norm_bwd(x[-5:].clone(), w, alone)
    assert torch.equal(g["dx"][-5:], h["dx"])
    torch.testing.assert_close(g["dweight"], h["dweight"], rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_eight_bits_are_of_the_quotient(dtype):
    """Rows whose scale is no power of two: every quotient of two 8-bit mantissas, rounded as the type does from the fp32
    quotient (103.5 of a row whose largest is 138 is a tie, 336, and goes to 320)."""
    import torch
    import recurrent_sequence_models_amd as rsm
    m = torch.arange(128, 256, dtype=torch.float32)
    x = torch.cat([m[:, None], torch.cat([m * 2.0 ** -e for e in range(1, 5)]).expand(128, -1), torch.zeros(128, 7)], 1)
    x[:, -7] = torch.where(m >= 138, 103.5, 0.0)
    scale = m / 448
    want = (x / scale[:, None]).to(torch.float8_e4m3fn).float()
    q, got = rsm.quantize_rows(x.to(dict(bf16=torch.bfloat16, fp32=torch.float32)[dtype]).cuda())
    assert torch.equal(got.cpu(), scale) and torch.equal(q.float().cpu(), want)
    assert want[10, -7] == 320
