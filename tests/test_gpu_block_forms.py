"""GPU tests of the block operators' forms at the sizes of block_cases: every tile of a product by rows and by columns,
ragged in each direction, on whole numbers (whose sums are exact in every form, so a product has one right answer), and
with activations and numbers between; the scan with many workgroups, and the convolution with its longest runs."""

import numpy as np
import pytest

import test_gpu_causal_conv as conv
import test_gpu_linear as lin
import test_gpu_selective_scan as scan
from block_cases import BACKWARD, CONV, CONV_NARROW, FORWARD, SCAN, scan_lens
from block_helpers import TINY, U, check, f64, half, offsets, rand, strided
from oracle import block as O

pytestmark = pytest.mark.gpu


def whole(seed, *shape, dtype, most=2):
    """Whole numbers from -most to most: products up to 4, of which even 16 400 add to less than 2^24, and whose sums
    lose nothing 13 bits behind the largest."""
    import torch
    a = np.random.Generator(np.random.PCG64(seed)).integers(-most, most + 1, size=shape)
    return torch.from_numpy(a.astype(np.float32)).to(dict(bf16=torch.bfloat16, fp32=torch.float32, e4m3=torch.float8_e4m3fn)[dtype]).cuda()


def view(t):
    import torch
    return strided(t.view(torch.uint8), 32).view(t.dtype) if t.dtype is torch.float8_e4m3fn else strided(t)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp32", "fp32"), ("e4m3", "bf16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("M,K,N", [s for s, _ in FORWARD])
def test_whole_numbers(dtype, out, M, K, N):
    import torch
    import recurrent_sequence_models_amd as rsm
    x, w = whole(1, M, K, dtype=dtype), whole(2, N, K, dtype=dtype)
    b, r = whole(3, N, dtype="fp32", most=9), whole(4, M, N, dtype=out, most=9)
    kw, p = {}, x.double() @ w.double().T
    if dtype == "e4m3":
        sx, sw = (2.0 ** whole(s, n, dtype="fp32", most=1) for s, n in ((5, M), (6, N)))
        kw = dict(x_scale=sx, weight_scale=sw, out_dtype=r.dtype)
        p = p * sx.double()[:, None] * sw.double()
    p = p + b
    want = (p + r).to(r.dtype)
    y, none = rsm.linear(view(x), w, bias=b, residual=r, **kw)
    assert none is None and torch.equal(y, want)
    z, pre = rsm.linear(x, w, bias=b, residual=r, pre=True, **kw)
    assert torch.equal(z, want) and torch.equal(pre, p.float())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K,N", [s for s, _ in BACKWARD])
def test_gradients_of_whole_numbers(dtype, M, K, N):
    import torch
    import recurrent_sequence_models_amd as rsm
    x, w, dy = whole(1, M, K, dtype=dtype), whole(2, N, K, dtype=dtype), whole(3, M, N, dtype=dtype)
    room = torch.full((M + 2, K + 16), 7.0, dtype=x.dtype, device="cuda")
    g = rsm.linear_bwd(view(x), w, view(dy), bias=True, dx=room[:M, :K])
    assert torch.equal(g["dx"], (dy.double() @ w.double()).to(x.dtype))
    assert torch.all(room[M:] == 7) and torch.all(room[:, K:] == 7)
    assert torch.equal(g["dweight"], (dy.double().T.contiguous() @ x.double()).to(x.dtype))
    assert torch.equal(g["dbias"], dy.double().sum(0).float())


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_large_ragged_tiles(dtype, out, act):
    """Of 256 x 256, the epilogue and numbers between whole ones."""
    lin.forward(dtype, 3996, 144, 4000, act, True, act == "silu", view=True, out=out)


@pytest.mark.parametrize("M,K,N", [s for s, _ in FORWARD if s[1] < 1000] + [(65, 2048, 264)])
def test_eight_bit_products(M, K, N):
    """Results in bf16 of the matrix unit's own 8-bit products, which no kept pre-activation asks to widen.  Bound: as in
    test_gpu_linear, 2^-13 of a row pair's largest product for each of K."""
    import torch
    import recurrent_sequence_models_amd as rsm
    (x, sx), (w, sw) = rsm.quantize_rows(rand(1, M, K)), rsm.quantize_rows(rand(2, N, K, scale=K ** -0.5))
    b, r = rand(3, N), rand(4, M, N, dtype="bf16")
    y, _ = rsm.linear(view(x), w, x_scale=sx, weight_scale=sw, bias=b, residual=r, activation="gelu")
    assert y.dtype is torch.bfloat16
    X, W, B, R = f64(x.float()) * f64(sx)[:, None], f64(w.float()) * f64(sw)[:, None], f64(b), f64(r)
    want, p = O.linear(X, W, B, "gelu", R)
    ep = (K + 32) * U * (np.abs(X) @ np.abs(W).T) + 4 * U * (np.abs(p) + np.abs(B))
    ep += K * 2.0 ** -13 * np.abs(X).max(-1)[:, None] * np.abs(W).max(-1)
    ey = 1.13 * ep + lin.act_error(p, want - R, "gelu") + 2 * U * (np.abs(want) + np.abs(R))
    check("y", f64(y), want, ey * (1 + half("bf16")) + half("bf16") * np.abs(want) + TINY)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("name", SCAN)
def test_scan_of_many_workgroups(name, N, dtype):
    """y, the final states and the gradients, which start from the states that this form keeps."""
    _, D, packed, _ = SCAN[name]
    lens = scan_lens(name, N)
    lead = (sum(lens),) if packed else (len(lens), lens[0])
    a = scan.inputs(1, lead, len(lens), D, N, dtype)
    scan.compare(a, lens, dtype, True, scan.run(a, offsets(lens) if packed else None, True, view=dtype == "fp32"))


@pytest.mark.parametrize("dtype,taps,act,D,lens", CONV)
def test_longest_runs_of_the_convolution(dtype, taps, act, D, lens):
    conv.both(conv.calls(act, view=dtype == "fp32"), dtype, lens, D, taps, act, init=True, view=dtype == "fp32")


@pytest.mark.parametrize("dtype,taps,act,D,lens", CONV_NARROW)
def test_narrow_convolution(dtype, taps, act, D, lens):
    conv.both(conv.calls(act, view=dtype == "fp32"), dtype, lens, D, taps, act, init=True, view=dtype == "fp32")
