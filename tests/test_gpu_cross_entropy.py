"""Softmax cross entropy on a linear layer and its gradient against the formulas in 64 bits: thin layers, few rows, tiles of
every size, pieces of classes and slabs of rows, operands that have to be packed, labels outside the classes, classes and
rows that are masked, magnitudes; the gradient against differences.

Tolerances, u = 2^-24, w the unit roundoff of the stored type. z is a sum of n terms in fp32: dz = (8 + 4 sqrt(n)) u S with S
the sum of its terms' magnitudes, as in the linear layer's tests. An exponential of x is off by (2 |x| + 8) u of itself
(its argument's rounding, twice, and 2^-21 for the approximation), a sum of k of them by (8 + 4 sqrt(k)) u. So
    lse    sum_j p_j dz_j + (8 + 4 sqrt(k) + 2 sum_j p_j (top - z_j)) u + 2 u (|lse| + |top|)
    loss   that, dz of the label's entry and 2 u of what is subtracted
    D      |g| p (dz + (2 |z - lse| + 8) u + 2 u |lse|) + 3 u |D| (lse is given), and w |D| where it is rounded; float16's D loses
           2^-25 / up at most, up the power of two that it is held at: 2^-39 of the largest |g|
Exponentials below fp32's smallest normal number come out as zero, and so do such entries of D and such sums: 2^-126 |g| of D and
2^-126 of a result are allowed for it. A product with D carries dD times the other operand's magnitudes, its own sum's (8 + 4 sqrt(K)) u S, and w of the result.
"""
import math

import pytest
import torch

import dense_linear_algebra_gb300 as fx

pytestmark = pytest.mark.gpu

U = 2.0**-24
W_OF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
FLUSH = 2.0**-126
TINY = {torch.float32: FLUSH, torch.bfloat16: FLUSH, torch.float16: 2.0**-25}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(shape, dtype, seed, scale=1.0, pad=0, offset=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)
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


def inputs(m, n, k, dtype, bias=True, w_t=True, pad=0, offset=0, spread=2.0, seed=0):
    X = make((m, n), dtype, seed + 1, pad=pad, offset=offset)
    W = make((k, n) if w_t else (n, k), dtype, seed + 2, spread / math.sqrt(n), pad, offset)
    W = W.t() if w_t else W
    b = make((1, k), dtype, seed + 3)[0] if bias else None
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 4)
    labels = torch.randint(0, k, (m,), generator=gen, device="cuda")
    drop = torch.rand(m, generator=gen, device="cuda")
    labels = torch.where(drop < 0.1, torch.where(drop < 0.05, -100, k), labels)
    if m:
        labels[0], labels[-1] = k - 1, 0
    return X, W, b, labels


def logits64(X, W, b):
    x, w = X.double(), W.double()
    z, S = x @ w, x.abs() @ w.abs()
    if b is not None:
        z, S = z + b.double(), S + b.double().abs()
    return z, S


def check(m, n, k, dtype, g=None, need=(True, True, True), edit=None, **kw):
    X, W, b, labels = inputs(m, n, k, dtype, **kw)
    if edit is not None:
        edit(X, W, b, labels)
    z, S = logits64(X, W, b)
    finite = torch.isfinite(z)
    dz = torch.where(finite, (8 + 4 * math.sqrt(n)) * U * S, 0.0)
    del S
    top, lse = z.max(1).values, torch.logsumexp(z, 1)
    inside = (labels >= 0) & (labels < k)
    at = torch.where(inside, labels, 0)[:, None]
    loss_got, lse_got = fx.cross_entropy(X, W, labels, b)
    again = fx.cross_entropy(X, W, labels.int(), b)
    p = torch.exp(z - lse[:, None])
    below = torch.where(p > 0, top[:, None] - z, 0.0)
    d_lse = 1.01 * (p * dz).sum(1) + (8 + 4 * math.sqrt(k) + 2 * (p * below).sum(1)) * U + 2 * U * (lse.abs() + top.abs())
    del below
    within(lse_got, lse, d_lse, "lse")
    loss = torch.where(inside, lse - z.gather(1, at)[:, 0], 0.0)
    d_loss = torch.where(inside, d_lse + dz.gather(1, at)[:, 0] + 2 * U * (loss.abs() + (top - z.gather(1, at)[:, 0]).abs()), 0.0)
    within(loss_got, loss, d_loss, "loss")
    assert torch.equal(loss_got, again[0]) and torch.equal(lse_got, again[1])

    if g is None:
        gen = torch.Generator(device="cuda")
        gen.manual_seed(9)
        g = torch.randn(m, generator=gen, device="cuda") / m
    lse32 = lse.float()
    got = fx.cross_entropy_grad(X, W, labels, lse32, b, g=g, need=need)
    again = fx.cross_entropy_grad(X, W, labels, lse32, b, g=g, need=need)
    torch.cuda.synchronize()
    assert fx.device_error() == fx.FXTX_OK
    assert [t is not None for t in got] == list(need)
    rows = torch.where(inside, g.double() if torch.is_tensor(g) else float(torch.tensor(g, dtype=torch.float32)), 0.0)
    p = torch.exp(z - lse32.double()[:, None])
    dD = rows.abs()[:, None] * p * (dz + (2 * torch.where(p > 0, (z - lse32.double()[:, None]).abs(), 0.0) + 8) * U + 2 * U * lse32.double().abs()[:, None])
    del z, dz
    D = p.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0)) * rows[:, None]
    del p
    dD += 3 * U * D.abs() + FLUSH * (1 + rows.abs().max())
    rounded = dD + (W_OF[dtype] * D.abs() if dtype is not torch.float32 else 0.0)
    if dtype is torch.float16:
        rounded += 2.0**-39 * rows.abs().max()
    x, w = X.double(), W.double()

    def product(got, want, S, loss, K, again, what):
        tol = (8 + 4 * math.sqrt(K)) * U * S + loss
        if dtype is torch.float16:  # from 65,520 on, halfway from its largest number to the next step, float16 rounds to infinity
            beyond = (want.abs() + tol * 1.01 >= 65_520) & torch.isinf(got) & (got.sign() == want.sign())
            got, want = torch.where(beyond, 0, got), torch.where(beyond, 0, want)
            again = torch.where(beyond, 0, again)
        within(got, want, tol + W_OF[dtype] * (want.abs() + tol) + TINY[dtype], what)
        assert torch.equal(got, again), what

    if need[0]:
        product(got[0], D @ w.t(), D.abs() @ w.abs().t(), rounded @ w.abs().t(), k, again[0], "dX")
        assert not got[0][~inside].any()
    if need[1]:
        product(got[1], x.t() @ D, x.abs().t() @ D.abs(), x.abs().t() @ rounded, m, again[1], "dW")
        assert min(n, k) == 1 or got[1].stride() == W.stride() or kw.get("pad")  # (with one of them, both orders are one)
    if need[2]:
        product(got[2], D.sum(0), D.abs().sum(0), dD.sum(0), m, again[2], "db")


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k", [(1, 1), (1, 2), (8, 3), (16, 16), (17, 10), (32, 10), (32, 17), (32, 32), (33, 33), (64, 10), (10, 64), (64, 64),
                                 (47, 61)])
def test_thin(n, k, dtype, w_t):
    check(1001, n, k, dtype, w_t=w_t, bias=n % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 64, 65, 5000, 100_003])
def test_thin_rows(m, dtype):
    check(m, 32, 10, dtype)
    check(m, 40, 20, dtype, g=1.0 / m)


SHAPES = [(1, 65, 1), (1, 1, 65), (3, 70, 130), (8, 100, 1000), (9, 100, 300), (16, 256, 999), (17, 256, 999), (100, 64, 65), (127, 130, 128),
          (128, 128, 256), (129, 200, 257), (300, 1001, 503), (257, 72, 5000), (1000, 513, 66), (2000, 96, 1000), (70, 2056, 2049)]


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(m, n, k, dtype, w_t):
    check(m, n, k, dtype, w_t=w_t, bias=(m + k) % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1)])
def test_column_slices(pad, offset, w_t, dtype):
    for m, n, k in ((200, 264, 1000), (12, 264, 1000), (500, 24, 16)):
        check(m, n, k, dtype, w_t=w_t, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, True, False)])
def test_parts_of_the_gradient(need, dtype):
    for m, n, k in ((300, 200, 700), (10, 200, 700), (900, 40, 50), (900, 64, 64)):
        check(m, n, k, dtype, need=need)


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_pieces_and_slabs(dtype, w_t):
    """More rows and more classes than one piece of D takes: sums over both."""
    check(17_000, 72, 33_000 if dtype is not torch.float32 else 17_000, dtype, w_t=w_t, bias=not w_t)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_of_few_classes(dtype):
    check(300_000, 80, 300, dtype, g=1.0 / 300_000)


@pytest.mark.parametrize("dtype", TYPES)
def test_packed_pieces(dtype):
    """Operands that the tensor copies cannot read, of more than one piece each."""
    check(140_000, 1001, 70, dtype, need=(False, True, False))
    check(30, 1001, 140_001, dtype, need=(True, False, False), w_t=False, pad=1, offset=0)


def test_long_features():
    """More than 8,192 features: sums in pieces."""
    check(300, 9000, 130, torch.bfloat16)
    check(130, 9000, 300, torch.float16, w_t=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(200, 40, 20), (5, 100, 900), (200, 100, 900)])
@pytest.mark.parametrize("masked", ["inf", "lowest"])
def test_masked_classes(m, n, k, dtype, masked):
    """Classes that a bias takes out, the first and last tile's among them; with -inf also those of some labels' rows."""
    low = float("-inf") if masked == "inf" else torch.finfo(dtype).min

    def edit(X, W, b, labels):
        b[: k // 3] = low
        b[k - k // 4:] = low
        labels.copy_(torch.where((labels >= 0) & (labels < k), k // 3 + labels % (k // 4), labels))

    check(m, n, k, dtype, edit=edit)


@pytest.mark.parametrize("m,n,k", [(200, 40, 20), (5, 100, 900), (200, 100, 900)])
def test_a_masked_label_and_no_class_left(m, n, k):
    X, W, b, labels = inputs(m, n, k, torch.float32)
    b[3] = float("-inf")
    labels[1] = 3
    loss, lse = fx.cross_entropy(X, W, labels, b)
    assert loss[1] == float("inf") and torch.isfinite(lse).all()
    dX, dW, db = fx.cross_entropy_grad(X, W, labels, lse, b, g=0.5)
    assert torch.isfinite(dX).all() and torch.isfinite(dW).all()
    assert abs(float(db[3]) + 0.5 * int((labels == 3).sum())) < 1e-5
    b[:] = float("-inf")
    loss, lse = fx.cross_entropy(X, W, labels, b)
    inside = (labels >= 0) & (labels < k)
    assert (lse == float("-inf")).all() and torch.isnan(loss[inside]).all() and not loss[~inside].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(100, 40, 20), (6, 100, 300), (100, 100, 300)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite(m, n, k, dtype, bad):
    """They make their own loss and gradient NaN; left out, they leave nothing in db and in other rows."""
    X, W, b, labels = inputs(m, n, k, dtype)
    labels.clamp_(0, k - 1)
    want = fx.cross_entropy(X, W, labels, b)
    dX, _, db = fx.cross_entropy_grad(X, W, labels, want[1], b, g=0.25)
    Y = X.clone()
    Y[2, 3] = bad
    got = fx.cross_entropy(Y, W, labels, b)
    keep = torch.arange(m, device="cuda") != 2
    assert torch.isnan(got[0][2]) and torch.isnan(got[1][2])
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    labels2 = labels.clone()
    labels2[2] = -1
    loss, _ = fx.cross_entropy(Y, W, labels2, b)
    assert loss[2] == 0
    dY, _, db2 = fx.cross_entropy_grad(Y, W, labels2, got[1], b, g=0.25)
    assert torch.equal(dY[keep], dX[keep]) and not dY[2].any() and torch.isfinite(db2).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spread", [1e-3, 30.0, 300.0])
@pytest.mark.parametrize("m,n,k", [(200, 40, 20), (8, 100, 900), (200, 100, 900)])
def test_spreads(m, n, k, dtype, spread):
    check(m, n, k, dtype, spread=spread)


@pytest.mark.parametrize("m,n,k", [(200, 40, 20), (200, 100, 5000)])
@pytest.mark.parametrize("g", [1e-7, 1e-12, 3e4, 0.0])
def test_float16_of_small_and_large_weights(m, n, k, g):
    """D keeps its digits where g lies far below float16's range; results are rounded to it."""
    X, W, b, labels = inputs(m, n, k, torch.float16)
    _, lse = fx.cross_entropy(X, W, labels, b)
    check(m, n, k, torch.float16, g=g)
    weights = torch.full((m,), g, device="cuda")
    a = fx.cross_entropy_grad(X, W, labels, lse, b, g=g)
    c = fx.cross_entropy_grad(X, W, labels, lse, b, g=weights)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


def test_no_rows():
    for n, k in ((100, 300), (20, 10)):
        X, W = torch.empty((0, n), device="cuda"), make((n, k), torch.float32, 1)
        labels = torch.empty(0, dtype=torch.int64, device="cuda")
        loss, lse = fx.cross_entropy(X, W, labels)
        assert loss.shape == (0,) and lse.shape == (0,)
        dX, dW, db = fx.cross_entropy_grad(X, W, labels, lse)
        assert dX.shape == (0, n) and not dW.any() and not db.any()


def test_gradient_against_differences():
    for m, n, k in ((12, 20, 9), (5, 70, 30), (20, 70, 30)):
        X, W, b, labels = inputs(m, n, k, torch.float32, w_t=False)
        g, step = torch.rand(m, device="cuda"), 1e-2
        _, lse = fx.cross_entropy(X, W, labels, b)
        grads = fx.cross_entropy_grad(X, W, labels, lse, b, g=g)
        args = [X, W, b]
        for i, grad in enumerate(grads):
            for at in range(0, args[i].numel(), max(1, args[i].numel() // 9)):
                moved = []
                for sign in (1, -1):
                    a = [t.clone() for t in args]
                    a[i].view(-1)[at] += sign * step
                    moved.append(float((fx.cross_entropy(a[0], a[1], labels, a[2])[0].double() * g.double()).sum()))
                # off by step^2 / 6 times the third derivative (sums of at most 20 terms below 20), and 1e-5 / step of fp32
                assert abs((moved[0] - moved[1]) / (2 * step) - float(grad.reshape(-1)[at])) < 70 * step**2 + 3e-3


def test_streams_and_graphs():
    for m, n, k, dtype in ((300, 200, 700, torch.bfloat16), (6, 200, 700, torch.float32), (900, 24, 10, torch.float16)):
        X, W, b, labels = inputs(m, n, k, dtype)
        side = torch.cuda.Stream()
        want = fx.cross_entropy(X, W, labels, b)
        want += fx.cross_entropy_grad(X, W, labels, want[1], b, g=1 / m)
        side.wait_stream(torch.cuda.current_stream())
        got = fx.cross_entropy(X, W, labels, b, stream=side)
        got += fx.cross_entropy_grad(X, W, labels, got[1], b, g=1 / m, stream=side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = fx.cross_entropy(X, W, labels, b)
            got += fx.cross_entropy_grad(X, W, labels, got[1], b, g=1 / m)
        X2, _, _, labels2 = inputs(m, n, k, dtype, seed=50)
        X.copy_(X2)
        labels.copy_(labels2)
        want = fx.cross_entropy(X, W, labels, b)
        want += fx.cross_entropy_grad(X, W, labels, want[1], b, g=1 / m)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
