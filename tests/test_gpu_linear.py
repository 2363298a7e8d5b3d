"""GPU tests of the projections with their epilogues, in bf16, fp32 and on 8-bit operands, and of their
gradients, elementwise against the fp64 definition.

Bounds, with u = 2^-24: a sum of K products is off by (K + 32) u of the sum of absolute values; scales and
bias add 4 u; the activations' slopes are at most 1.13 and their second derivatives at most 1; silu is off by
(2 |p| + 10) u |y| more, gelu by 8 u |p| (1 + erf cancels); results are rounded once (half).  In the backward
pass the products of bf16 take d rounded once (half).  The 8-bit products of the matrix unit, used for
bf16 results (not always for up to 64 tokens, nor with a kept pre-activation), drop what lies 13 bits behind the largest product of a
group: up to 2^-13 of the largest product of the row pair for each of K."""

import numpy as np
import pytest

from block_helpers import TINY, U, check, f64, half, rand, same_in_graph, strided
from oracle import block as O

pytestmark = pytest.mark.gpu

# few tokens (1 to 64: 1, 2 and 4 blocks of 16, or tiles), tiles of 64 with k split and not, of 128; ragged in each direction
SIZES = [(1, 16, 8), (7, 48, 24), (16, 2048, 72), (17, 176, 200), (33, 4096, 136), (64, 80, 1000), (65, 16, 8), (100, 1040, 40),
         (129, 2048, 264), (500, 64, 640), (3000, 208, 1288)]
BIG = (4100, 144, 4000)      # 33 x 32 tiles of 128, two a compute unit; 4096 tokens on 4096 make 16 x 16 of 256
# 256 tiles of 128; 32 and 64 of them with k in 8 parts; one in 16 (longer rows than quantize_rows takes)
MIDDLE, LONG = [(2040, 272, 2040), (1000, 16384, 512), (1000, 8208, 1016)], (70, 100384, 72)
# the same for dx, for dweight, and for dweight in parts
MIDDLE_BACK = [(2040, 2032, 264), (300, 2032, 2040), (8200, 1008, 1000)]


def act_error(p, y, act):
    if act == "silu":
        return np.abs(y) * (2 * np.abs(p) + 10) * U
    return 8 * U * np.abs(p) if act == "gelu" else 0.0


def quantised(t):
    import recurrent_sequence_models_amd as rsm
    return rsm.quantize_rows(t)


def forward(dtype, M, K, N, act, bias, residual, view=False, out=None):
    import torch
    import recurrent_sequence_models_amd as rsm
    dt = "fp32" if dtype == "e4m3" else dtype
    x, w = rand(1, M, K, dtype=dt), rand(2, N, K, dtype=dt, scale=K ** -0.5)
    kw = {}
    X, W = f64(x), f64(w)
    ydt = dt if out is None else out
    if dtype == "e4m3":
        (x, sx), (w, sw) = quantised(x), quantised(w)
        kw = dict(x_scale=sx, weight_scale=sw, out_dtype={"bf16": torch.bfloat16, "fp32": torch.float32}[ydt])
        X, W = f64(x.float()) * f64(sx)[:, None], f64(w.float()) * f64(sw)[:, None]
    b = rand(3, N) if bias else None
    r = rand(4, M, N, dtype=ydt) if residual else None
    xv = strided(x.view(torch.uint8), 32).view(x.dtype) if view and dtype == "e4m3" else strided(x) if view else x
    y, pre = rsm.linear(xv, w, bias=b, activation=act, residual=r, pre=True, **kw)
    B, R = (0.0 if t is None else f64(t) for t in (b, r))
    want, p = O.linear(X, W, B, act, R)
    ep = (K + 32) * U * (np.abs(X) @ np.abs(W).T) + 4 * U * (np.abs(p) + np.abs(B))
    if dtype == "e4m3" and ydt == "bf16":
        ep = ep + K * 2.0 ** -13 * (np.abs(X)[:, None] * np.abs(W)[None]).max(-1) if M * K * N < 1 << 28 else \
            ep + K * 2.0 ** -13 * np.abs(X).max(-1)[:, None] * np.abs(W).max(-1)
    check("pre", f64(pre), p, ep + TINY)
    ey = 1.13 * ep + act_error(p, want - R, act) + 2 * U * (np.abs(want) + np.abs(R))
    check("y", f64(y), want, ey * (1 + half(ydt)) + half(ydt) * np.abs(want) + TINY)


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("act,bias,residual,view", [(None, False, False, False), ("silu", True, True, True), ("gelu", True, False, False)])
def test_forward(dtype, M, K, N, act, bias, residual, view):
    forward(dtype, M, K, N, act, bias, residual, view, out="bf16" if dtype == "e4m3" and act else None)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("M,K,N", [BIG, (4099, 512, 4096), (4096 + 64, 512, 4096)])
def test_large_tiles(dtype, out, M, K, N):
    """Also with a few tokens behind the last whole tile, which a pass of their own takes."""
    forward(dtype, M, K, N, "silu", True, True, view=True, out=out)


@pytest.mark.parametrize("dtype,out,M,K,N", [(d, o, *size) for d, o in (("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "fp32"), ("fp32", "fp32"))
                                             for size in MIDDLE + [LONG] * (d != "e4m3")])
def test_middle_tiles(dtype, out, M, K, N):
    forward(dtype, M, K, N, None, True, False, view=True, out=out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K,N", SIZES + [(1, 64, 4096), (5000, 48, 72), (777, 1536, 384)])
@pytest.mark.parametrize("act,view", [(None, False), ("silu", True), ("gelu", False)])
def test_backward(dtype, M, K, N, act, view):
    backward(dtype, M, K, N, act, view)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K,N", MIDDLE_BACK)
def test_middle_tiles_backward(dtype, M, K, N):
    backward(dtype, M, K, N, None, True)


def backward(dtype, M, K, N, act, view):
    import torch
    import recurrent_sequence_models_amd as rsm
    x, w, b, dy = rand(1, M, K, dtype=dtype), rand(2, N, K, dtype=dtype, scale=K ** -0.5), rand(3, N), rand(5, M, N, dtype=dtype)
    _, pre = rsm.linear(x, w, bias=b, activation=act, pre=act is not None)
    P = f64(pre) if act else np.zeros((M, N))
    dxv = strided(torch.empty_like(x)) if view else True
    g = rsm.linear_bwd(strided(x) if view else x, w, strided(dy) if view else dy, pre=pre, activation=act, bias=True, dx=dxv)
    X, W, DY = f64(x), f64(w), f64(dy)
    ref = O.linear_backward(X, W, DY, P, act)
    ed = (np.abs(DY) * 16 * U * (1 + np.abs(P)) + half(dtype) * np.abs(ref["d"]) + TINY) if act else 0 * DY
    size = np.abs(ref["d"]) + ed
    check("dx", f64(g["dx"]), ref["dx"], ed @ np.abs(W) + (N + 32) * U * (size @ np.abs(W)) + half(dtype) * np.abs(ref["dx"]) + TINY)
    check("dweight", f64(g["dweight"]), ref["dw"],
          ed.T @ np.abs(X) + (M + 32) * U * (size.T @ np.abs(X)) + half(dtype) * np.abs(ref["dw"]) + TINY)
    eb = np.abs(DY) * 16 * U * (1 + np.abs(P)) if act else 0 * DY
    check("dbias", f64(g["dbias"]), ref["db"], (eb + (min(M, 200) + 100) * U * np.abs(ref["d"])).sum(0) + TINY)
    assert g["dx"].dtype is x.dtype and g["dweight"].dtype is x.dtype
    only = rsm.linear_bwd(x, w, dy, pre=pre, activation=act, dx=False)
    assert only["dx"] is None and only["dbias"] is None and torch.equal(only["dweight"], g["dweight"])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_are_those_of_differences(act):
    r = np.random.default_rng(1)
    x, w, b, dy = r.normal(size=(5, 7)), r.normal(size=(4, 7)), r.normal(size=4), r.normal(size=(5, 4))
    g = O.linear_backward(x, w, dy, O.linear(x, w, b)[1], act)
    args = [x, w, b]
    for i, k in enumerate(("dx", "dw", "db")):
        d, h = r.normal(size=args[i].shape), 1e-6
        f = lambda t: (dy * O.linear(*[a + t * d if i == j else a for j, a in enumerate(args)], act)[0]).sum()  # noqa: E731
        assert abs((f(h) - f(-h)) / (2 * h) - (g[k] * d).sum()) < 1e-7


@pytest.mark.parametrize("M", [5, 150])
def test_far_arguments_and_no_numbers(M):
    """Activations far out, and infinities and NaN that stay in their rows and columns."""
    import torch
    import recurrent_sequence_models_amd as rsm
    K, N = 80, 72
    x, w = rand(1, M, K, dtype="bf16"), rand(2, N, K, dtype="bf16")
    b = torch.zeros(N, device="cuda")
    b[0], b[1] = 1e30, -1e30
    for act in ("silu", "gelu"):
        y, _ = rsm.linear(x, w, bias=b, activation=act)
        assert torch.isfinite(y).all() and (y[:, 0] > 9e29).all() and (y[:, 1] == 0).all()
    good, _ = rsm.linear(x, w)
    bad, wb = x.clone(), w.clone()
    bad[3, 5], bad[1, K - 1], wb[7, 0] = float("inf"), float("nan"), float("nan")
    y, _ = rsm.linear(bad, wb)
    rows = [i for i in range(M) if i not in (1, 3)]
    cols = [i for i in range(N) if i != 7]
    assert torch.equal(y[rows][:, cols], good[rows][:, cols])
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 7]).all() and not torch.isfinite(y[3]).any()
    g0, g1 = rsm.linear_bwd(x, w, good), rsm.linear_bwd(bad, w, good)
    assert torch.equal(g0["dx"], g1["dx"])                             # does not read x
    keep = [i for i in range(K) if i not in (5, K - 1)]
    assert torch.equal(g0["dweight"][:, keep], g1["dweight"][:, keep])


def test_in_place_graphs_and_streams():
    import torch
    import recurrent_sequence_models_amd as rsm
    M, K, N = 300, 2048, 136
    x, w, b, r = rand(1, M, K, dtype="bf16"), rand(2, N, K, dtype="bf16"), rand(3, N), rand(4, M, N, dtype="bf16")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    (xq, sx), (wq, sw) = rsm.quantize_rows(x), rsm.quantize_rows(w)

    def call(stream=None):
        kw = dict(workspace=ws, stream=stream)
        y, pre = rsm.linear(x, w, bias=b, activation="silu", residual=r, pre=True, **kw)
        few, _ = rsm.linear(x[:9], w, bias=b, **kw)
        q, _ = rsm.linear(xq, wq, x_scale=sx, weight_scale=sw, bias=b, **kw)
        g = rsm.linear_bwd(x, w, y, pre=pre, activation="silu", bias=True, **kw)
        return [y, pre, few, q, *g.values()]
    want = call()
    z = r.clone()
    y, _ = rsm.linear(x, w, bias=b, activation="silu", residual=z, out=z)
    assert y is z and torch.equal(z, want[0])
    room = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    rsm.linear(x, w, bias=b, activation="silu", residual=r, out=room[:M])
    assert torch.equal(room[:M], want[0]) and torch.all(room[M:] == 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    same_in_graph(call)


def test_past_32_bits():
    """Rows of x and y behind 2^31 entries, and tokens 2^23 bytes apart."""
    import torch
    import recurrent_sequence_models_amd as rsm
    K, N, M = 2048, 2048, (1 << 20) + 70
    w, tail = rand(1, N, K, dtype="bf16"), rand(2, 70, K, dtype="bf16")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-70:] = tail
    y, _ = rsm.linear(x, w)
    want, _ = rsm.linear(tail, w)
    assert not y[:-70].any()
    torch.testing.assert_close(y[-70:].float(), want.float(), rtol=2 ** -7, atol=1e-3)
    g = rsm.linear_bwd(x, w, y, dweight=False)
    h = rsm.linear_bwd(tail, w, y[-70:].clone(), dweight=False)
    assert not g["dx"][:-70].any()
    torch.testing.assert_close(g["dx"][-70:].float(), h["dx"].float(), rtol=2 ** -6, atol=0.5)
    del x, y, g
    step, rows = 1 << 22, 300
    wide = torch.zeros(rows, step, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = rand(3, rows, K, dtype="bf16")
    y, _ = rsm.linear(wide[:, :K], w)
    z, _ = rsm.linear(wide[:, :K].contiguous(), w)
    assert torch.equal(y, z)


def test_one_token_over_its_bias():
    """One token's bias may be where its result goes: the threads that read it store there."""
    import torch
    import recurrent_sequence_models_amd as rsm
    for K, N in ((80, 72), (8208, 1016)):                    # 16 rows of W a workgroup, and tiles with k in parts
        x, w, b = rand(1, K), rand(2, N, K), rand(3, N)
        want, _ = rsm.linear(x, w, bias=b)
        y, _ = rsm.linear(x, w, bias=b, out=b)
        assert y is b and torch.equal(b, want)


# of 8-bit operands to bf16: tiles of 64 with k split and whole, of 128 (deep, two a unit), of 256 with tokens apart
@pytest.mark.parametrize("M,K,N", [(65, 2048, 264), (500, 80, 640), (2040, 272, 2040), (2050, 272, 2552), (4099, 144, 4096)])
def test_kept_pre_activation_of_8_bits(M, K, N):
    """The fp32 pre-activation is the sum in fp32, also where a result rounded to bf16 would not show more than 13 bits:
    beside one large product a group's others would be dropped.  Bound: of forward(), without that."""
    import torch
    import recurrent_sequence_models_amd as rsm
    g = torch.Generator(device="cuda").manual_seed(7)
    x, w = (2 + 3 * torch.rand(n, K, generator=g, device="cuda") for n in (M, N))     # products of 2^-14 of the largest
    x[:, ::64], w[:, ::64] = 448.0, 448.0
    x[1::2, ::64] *= -1
    x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    sx, sw, b = torch.rand(M, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") + 0.5, rand(3, N)
    y, pre = rsm.linear(x, w, x_scale=sx, weight_scale=sw, bias=b, activation="silu", pre=True)
    X, W, B = f64(x.float()) * f64(sx)[:, None], f64(w.float()) * f64(sw)[:, None], f64(b)
    want, p = O.linear(X, W, B, "silu")
    ep = (K + 32) * U * (np.abs(X) @ np.abs(W).T) + 4 * U * (np.abs(p) + np.abs(B))
    check("pre", f64(pre), p, ep + TINY)
    check("y", f64(y), want, (1.13 * ep + act_error(p, want, "silu")) * (1 + half("bf16")) + half("bf16") * np.abs(want) + TINY)
