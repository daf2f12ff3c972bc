"""Layer norm and its gradient against the formulas in 64 bits, over types, row lengths from one entry to those that the
registers do not hold, odd pitches, rows of one value, rows that are not finite; the gradient against differences.

Tolerances, u = 2^-24, w the unit roundoff of the stored type. A sum of a row's n terms is formed by at most 32 terms a
thread in turn, an exchange over 32 lanes and at most 32 warps in turn: 32 + 5 + 32 roundings, C = 80 with what the terms
themselves round. So mean is within C u avg|x|; the variance within C u of itself plus that error's square; u = (x -
mean) rstd within rstd times mean's error, 2 u |x - mean| for its own operations and half the variance's relative error.
Column sums are taken as in the linear layer's tests: (8 + 4 sqrt(m)) u of the sum of the terms' magnitudes.
"""
import math

import pytest
import torch

import dense_linear_algebra_gb300 as fx

pytestmark = pytest.mark.gpu

U = 2.0**-24
W_OF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0**-25}  # half the smallest float16
TYPES = [torch.bfloat16, torch.float16, torch.float32]
C = 80.0
EPS = 1e-5


def make(shape, dtype, seed, scale=1.0, shift=0.0, pad=0, offset=0):
    """A matrix of normal values; with `pad`, a column slice of a wider one (poisoned around it)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)
    if not pad:
        return x
    wide = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, offset:offset + shape[1]] = x
    return wide[:, offset:offset + shape[1]]


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {bad.nonzero()[0].tolist()}, worst "
                           f"{float((err / tol).nan_to_num(1e9).max()):.3g} of the tolerance")


def stats64(x, eps):
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, var, 1 / torch.sqrt(var + eps)


def check_forward(m, n, dtype, affine=True, scale=1.0, shift=0.0, pad=0, offset=0, eps=EPS, seed=0):
    X = make((m, n), dtype, seed + 1, scale, shift, pad, offset)
    w = make((1, n), dtype, seed + 2, 0.3, 1.0)[0] if affine else None
    b = make((1, n), dtype, seed + 3)[0] if affine else None
    out = make((m, n), dtype, seed + 4, pad=pad, offset=offset) if pad else None
    got, mean, rstd = fx.layer_norm(X, w, b, eps=eps, stats=True, out=out)
    again = fx.layer_norm(X, w, b, eps=eps)
    torch.cuda.synchronize()
    x = X.double()
    mean64, var, rstd64 = stats64(x, eps)
    e32 = float(torch.tensor(eps, dtype=torch.float32))
    d_mean = C * U * x.abs().mean(1)
    within(mean, mean64, d_mean, "mean")
    d_var = C * U * var + d_mean.square() + U * e32
    d_rstd = rstd64 * (0.5 * d_var / (var + eps) + 2 * U) * 1.01
    within(rstd, rstd64, d_rstd, "rstd")
    c = x - mean64[:, None]
    u = c * rstd64[:, None]
    d_u = rstd64[:, None] * (d_mean[:, None] + 2 * U * c.abs()) + c.abs() * d_rstd[:, None] * 1.01
    want = u * w.double() + b.double() if affine else u
    tol = d_u * (w.double().abs() if affine else 1.0) + 3 * U * u.abs() + W_OF[dtype] * want.abs() + TINY[dtype]
    if affine:
        tol = tol + 3 * U * ((u * w.double()).abs() + b.double().abs())
    within(got, want, tol * 1.001, "out")
    assert torch.equal(got, again)
    if pad:  # what lies beside the slice stays
        wide = got._base
        assert torch.isnan(wide[:, :offset]).all() and torch.isnan(wide[:, offset + n:]).all()


def check_grad(m, n, dtype, affine=True, residual=True, scale=1.0, shift=0.0, pad=0, offset=0, need=(True, True, True), seed=0):
    X = make((m, n), dtype, seed + 1, scale, shift, pad, offset)
    G = make((m, n), dtype, seed + 2, pad=pad, offset=offset)
    R = make((m, n), dtype, seed + 3, pad=pad, offset=offset) if residual else None
    w = make((1, n), dtype, seed + 4, 0.3, 1.0)[0] if affine else None
    x = X.double()
    mean, _, rstd = stats64(x, EPS)
    mean, rstd = mean.float(), rstd.float()
    dX, dw, db = fx.layer_norm_grad(G, X, w, mean, rstd, residual=R, need=need)
    again = fx.layer_norm_grad(G, X, w, mean, rstd, residual=R, need=need)
    torch.cuda.synchronize()
    g = G.double()
    u = (x - mean.double()[:, None]) * rstd.double()[:, None]
    h = g * w.double() if affine else g
    s = rstd.double()[:, None]
    c1, c2 = h.mean(1, keepdim=True), (h * u).mean(1, keepdim=True)
    want = s * (h - c1 - u * c2)
    tol = s * (6 * U * (h.abs() + c1.abs() + (u * c2).abs()) + C * U * (h.abs().mean(1, keepdim=True)
                                                                       + u.abs() * (h * u).abs().mean(1, keepdim=True)))
    if residual:
        want = want + R.double()
        tol = tol + U * R.double().abs()
    if need[0]:
        within(dX, want, tol + W_OF[dtype] * (want.abs() + tol) + TINY[dtype], "dX")
        assert torch.equal(dX, again[0])
    c = (8 + 4 * math.sqrt(max(m, 1))) * U
    for got, terms, other in ((dw, g * u, again[1]), (db, g, again[2])):
        if got is not None:
            total = terms.sum(0)
            within(got, total, c * terms.abs().sum(0) + W_OF[dtype] * total.abs() * 1.001 + TINY[dtype], "column sums")
            assert torch.equal(got, other)
    assert [t is not None for t in (dX, dw, db)] == list(need)


# one access a thread, several lanes, a warp, several warps, the most that registers hold and one more, by 16 bytes and by
# entries
LENGTHS = [1, 2, 3, 7, 8, 16, 31, 32, 33, 64, 100, 127, 128, 129, 256, 264, 301, 512, 513, 1000, 1001, 1024, 2056, 4096, 4104, 5000, 5912,
           6144, 8192, 8200, 8193, 16384, 16392, 32768, 32776]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", LENGTHS)
def test_forward_lengths(n, dtype):
    check_forward(5, n, dtype, affine=n % 3 != 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", LENGTHS)
def test_gradient_lengths(n, dtype):
    check_grad(7, n, dtype, affine=n % 3 != 0, residual=n % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(1, 4096), (2, 8), (513, 32), (1000, 40), (4097, 24), (100_003, 32), (3001, 301), (700, 4096), (65, 16384),
                                 (1217, 1024), (33, 40_000), (2500, 5)])
def test_rows(m, n, dtype):
    check_forward(m, n, dtype)
    check_grad(m, n, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(8001, 129), (8000, 250), (8003, 257), (6001, 511), (6000, 1001), (3001, 2047), (1500, 4099), (900, 8191), (9000, 130)])
def test_many_rows_of_odd_widths(m, n, dtype):
    """Rows that come by bulk copies from where they lie, whole 16 bytes around them; the last one's end is read apart."""
    check_forward(m, n, dtype, affine=n != 257, shift=1.0)
    check_grad(m, n, dtype, residual=m % 2 == 1, affine=n != 511, need=(True, n != 1001, n != 1001))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(400_001, 8), (200_003, 16), (100_001, 40), (100_003, 64), (50_001, 104), (30_011, 128), (20_003, 232)])
def test_many_short_rows(m, n, dtype):
    """Tiles of rows that come by bulk copies, the last one short."""
    check_grad(m, n, dtype, residual=m % 4 == 3, affine=n != 64, need=(True, n != 40, n != 40))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(5001, 1160), (6000, 2056), (3000, 4096), (1300, 5000), (1300, 8192), (700, 16384), (2500, 4104)])
def test_many_long_rows(m, n, dtype):
    """Rows that come by bulk copies."""
    check_forward(m, n, dtype, shift=3.0)
    check_grad(m, n, dtype, residual=n % 16 == 0, need=(True, n != 2056, n != 2056))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (1, 0), (5, 3)])
@pytest.mark.parametrize("m,n", [(9, 32), (9, 301), (9, 1024), (9, 20_000), (3000, 2048), (5000, 700)])
def test_column_slices(m, n, pad, offset, dtype):
    check_forward(m, n, dtype, pad=pad, offset=offset)
    check_grad(m, n, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,shift", [(1e-3, 0.0), (1e3, 0.0), (1.0, 30.0), (0.01, 1.0), (1e-6, 0.0)])
def test_magnitudes(scale, shift, dtype):
    check_forward(64, 777, dtype, scale=scale, shift=shift)
    check_forward(64, 1024, dtype, scale=scale, shift=shift)
    check_grad(64, 1024, dtype, scale=scale, shift=shift)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, True), (False, False, True), (False, True, False), (True, True, False)])
@pytest.mark.parametrize("n", [24, 1000, 17_000])
def test_parts_of_the_gradient(n, need):
    check_grad(300, n, torch.bfloat16, need=need)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_one_value(dtype):
    """Without spread a row comes out as the bias, and rstd is eps^-1/2."""
    X = torch.full((6, 640), 1.5, dtype=dtype, device="cuda")
    b = make((1, 640), dtype, 1)[0]
    out, mean, rstd = fx.layer_norm(X, None, b, stats=True)
    assert torch.equal(mean, torch.full_like(mean, 1.5))
    assert (rstd * math.sqrt(EPS) - 1).abs().max() < 4 * U
    assert torch.equal(out, b.expand(6, 640))
    out = fx.layer_norm(X[:, :1], None, None, eps=1e-12)
    assert torch.equal(out, torch.zeros_like(out))


def test_no_rows():
    X = torch.empty((0, 64), device="cuda")
    out, mean, rstd = fx.layer_norm(X, stats=True)
    assert out.shape == (0, 64) and mean.shape == (0,)
    dX, dw, db = fx.layer_norm_grad(X, X, None, mean, rstd)
    assert dX.shape == (0, 64) and torch.equal(dw, torch.zeros_like(dw)) and torch.equal(db, torch.zeros_like(db))
    X = torch.empty((0, 40_000), device="cuda")
    dX, dw, db = fx.layer_norm_grad(X, X, None, mean, rstd)
    assert torch.equal(dw, torch.zeros_like(dw)) and torch.equal(db, torch.zeros_like(db))


@pytest.mark.parametrize("n", [32, 1024, 4096, 40_000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite(n, bad):
    """They come out as NaN and leave the other rows alone."""
    X, G = make((10, n), torch.float32, 1), make((10, n), torch.float32, 2)
    want, mean, rstd = fx.layer_norm(X, stats=True)
    dX, _, db = fx.layer_norm_grad(G, X, None, mean, rstd)
    Y = X.clone()
    Y[3, 5] = bad
    out, mean, rstd = fx.layer_norm(Y, stats=True)
    keep = torch.arange(10, device="cuda") != 3
    assert torch.equal(out[keep], want[keep]) and torch.isnan(out[3, 5])
    got, _, db2 = fx.layer_norm_grad(G, Y, None, mean, rstd)
    assert torch.equal(got[keep], dX[keep]) and torch.isnan(got[3]).all()
    assert torch.equal(db, db2)


@pytest.mark.parametrize("n", [40, 1000, 4096, 40_000])
def test_in_place(n):
    X, G, R = (make((50, n), torch.bfloat16, s) for s in (1, 2, 3))
    want, mean, rstd = fx.layer_norm(X, stats=True)
    Y = X.clone()
    assert torch.equal(fx.layer_norm(Y, out=Y), want) and torch.equal(Y, want)
    dX, _, _ = fx.layer_norm_grad(G, X, None, mean, rstd, residual=R)
    for i in range(3):  # DX over G, over R, over X
        a = [G.clone(), X.clone(), R.clone()]
        rc = fx.fxtx_layer_norm_grad(1, 50, n, a[0].data_ptr(), n, a[1].data_ptr(), n, None, mean.data_ptr(), rstd.data_ptr(),
                                     a[2].data_ptr(), n, a[i].data_ptr(), n, None, None, torch.cuda.current_stream().cuda_stream)
        assert rc == fx.FXTX_OK and torch.equal(a[i], dX)


def test_gradient_against_differences():
    """Of sum(out * G), in float32 with steps that its rounding allows."""
    m, n, step = 4, 48, 1e-2
    X, G = make((m, n), torch.float32, 1), make((m, n), torch.float32, 2)
    w, b = make((1, n), torch.float32, 3)[0], make((1, n), torch.float32, 4)[0]

    def value(X, w, b):
        return float((fx.layer_norm(X, w, b).double() * G.double()).sum())

    _, mean, rstd = fx.layer_norm(X, w, b, stats=True)
    grads = fx.layer_norm_grad(G, X, w, mean, rstd)
    args = [X, w, b]
    for i, grad in enumerate(grads):
        for at in range(0, args[i].numel(), 7):
            moved = []
            for sign in (1, -1):
                a = [t.clone() for t in args]
                a[i].view(-1)[at] += sign * step
                moved.append(value(*a))
            # a central difference is off by step^2 / 6 times the third derivative, here below 10; fp32 adds 1e-5 / step
            assert abs((moved[0] - moved[1]) / (2 * step) - float(grad.view(-1)[at])) < 10 * step**2 + 2e-3


def test_streams_and_graphs():
    X, G = make((777, 520), torch.float16, 1), make((777, 520), torch.float16, 2)
    out, mean, rstd = fx.layer_norm(X, stats=True)
    grads = fx.layer_norm_grad(G, X, None, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fx.layer_norm(X, stats=True, stream=side)
    got2 = fx.layer_norm_grad(G, X, None, got[1], got[2], stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip((out, mean, rstd, *grads), (*got, *got2)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fx.layer_norm(X, stats=True)
        got2 = fx.layer_norm_grad(G, X, None, got[1], got[2])
    Y = make((777, 520), torch.float16, 3)
    want = fx.layer_norm(Y, stats=True)
    want2 = fx.layer_norm_grad(G, Y, None, want[1], want[2])
    X.copy_(Y)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*want, *want2), (*got, *got2)):
        assert torch.equal(a, b)
