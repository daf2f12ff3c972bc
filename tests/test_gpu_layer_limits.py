"""Layers at the ends of their ranges: sums over hundreds of thousands of terms of one sign, sums whose length comes close
to 2^31, float32 values that are not finite or tiny, and few float32 rows in slices."""
import pytest
import torch

import dense_linear_algebra_gb300 as fx
from test_gpu_linear import check_grad, check_linear

pytestmark = pytest.mark.gpu


def _positive(shape, dtype, seed, scale=1.0, spread=None):
    """Values of 1 to 2 times `scale`; `spread`: its rows (0) or columns (1) each times a factor of 1 to 2 of their own."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (torch.rand(shape, generator=gen, device="cuda") + 1) * scale
    if spread is not None:
        f = torch.rand(shape[spread], generator=gen, device="cuda") + 1
        x *= f[:, None] if spread == 0 else f
    return x.to(dtype)


def _bias(got, A, B, rows, cols):
    """The mean relative error of entries (rows, cols) of A^T B, in 64 bits, A and B taken a piece of their rows at a time."""
    want = torch.zeros(len(rows), len(cols), dtype=torch.float64, device="cuda")
    for at in range(0, A.shape[0], 100_000):
        want += A[at:at + 100_000][:, rows].double().t() @ B[at:at + 100_000][:, cols].double()
    return float((got[rows][:, cols].double() / want - 1).mean())


def _some(n):
    return torch.linspace(0, n - 1, min(n, 64)).long().cuda()


# Sums of positive terms: the tensor cores add 16 terms at a time to an accumulator, and drop what lies below its last
# bit: at most 2^-23 of it. If at most 16,384 terms stay there, 1,024 such steps leave at most 1024 * 2^-23 of half the sum (it
# grows evenly) on average, 2^-14, an eighth of float16's rounding. Roundings to the type average out over entries of 4,096 sizes:
# w over the square root of 3 * 4096, 2^-14.8 for bfloat16.
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("m,n,k", [(300_000, 4096, 2048), (400_001, 264, 200)])
def test_long_gradient_sums(m, n, k, dtype):
    X, G = _positive((m, n), dtype, 1, spread=1), _positive((m, k), dtype, 2, 1 / 128, spread=1)
    W = torch.zeros(n, k, dtype=dtype, device="cuda")
    _, dW, db = fx.linear_grad(G, X, W, need=(False, True, True))
    assert fx.device_error() == fx.FXTX_OK
    w = 2.0**-8 if dtype == torch.bfloat16 else 2.0**-11
    assert abs(_bias(dW, X, G, _some(n), _some(k))) <= 2.0**-14 + w / 4096**0.5
    assert float((db.double() / G.double().sum(0) - 1).abs().max()) <= 2.0**-14 + w


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("m,n,k", [(40, 1_000_000, 512), (1, 600_001, 96), (3000, 200_000, 2560)])
def test_long_layer_sums(m, n, k, w_t):
    dtype = torch.float16
    X, W = _positive((m, n), dtype, 3, 1 / 512, 0), _positive((k, n) if w_t else (n, k), dtype, 4, spread=0 if w_t else 1)
    W = W.t() if w_t else W
    got, Z = fx.linear(X, W, pre=True)
    assert fx.device_error() == fx.FXTX_OK
    assert torch.equal(got, Z)
    assert abs(_bias(got, X.t(), W, _some(m), _some(k))) <= 2.0**-14 + 2.0**-11 / (min(m, 64) * 64) ** 0.5


@pytest.mark.parametrize("m,n,k", [(200_000_000, 8, 8), (40_000_000, 40, 60)])
def test_long_thin_gradient_sums(m, n, k):
    """The same for at most 64 features and outputs, where a warp adds 16 rows at a time: the same 2^-14, and the roundings of n k entries."""
    X, G = _positive((m, n), torch.float16, 5, 2.0**-6, 1), _positive((m, k), torch.float16, 6, 2.0**-14, 1)
    _, dW, db = fx.linear_grad(G, X, torch.zeros(n, k, dtype=torch.float16, device="cuda"), need=(False, True, True))
    want, sums = torch.zeros(n, k, dtype=torch.float64, device="cuda"), torch.zeros(k, dtype=torch.float64, device="cuda")
    for at in range(0, m, 4_000_000):
        g = G[at:at + 4_000_000].double()
        want += X[at:at + 4_000_000].double().t() @ g
        sums += g.sum(0)
    assert abs(float((dW.double() / want - 1).mean())) <= 2.0**-14 + 2.0**-11 / (n * k) ** 0.5
    assert float((db.double() / sums - 1).abs().max()) <= 2.0**-14 + 2.0**-11


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 600])
def test_few_rows_of_nearly_2_31_features(n, w_t):
    """float32, one row: small whole numbers at both ends and in between, the sums exact."""
    X = torch.zeros(1, n, device="cuda")
    W = torch.zeros((2, n) if w_t else (n, 2), device="cuda")
    W = W.t() if w_t else W
    at = torch.cat([torch.arange(3), n // 8 * torch.arange(1, 8), torch.arange(n - 700, n, 7), torch.tensor([n - 1])]).cuda()
    X[0, at] = torch.arange(1, at.numel() + 1, device="cuda").float() % 13
    W[at, 0], W[at, 1] = 1.0, torch.arange(at.numel(), device="cuda").float() % 5
    got = fx.linear(X, W)
    assert torch.equal(got[0].double(), X[0, at].double() @ W[at].double())


@pytest.mark.parametrize("m,n,k", [(2, 200, 136), (6, 300, 200), (300, 200, 136), (300, 24, 40)])
@pytest.mark.parametrize("w_t", [False, True])
def test_float32_non_finite_stays_in_its_row(m, n, k, w_t):
    """Where a row of float32 holds an infinity or a NaN, nothing finite comes out of it, and the other rows are what they were:
    an infinity comes out as one or as a NaN (products of a value's three terms have no infinity)."""
    X, W = _positive((m, n), torch.float32, 5), _positive((k, n) if w_t else (n, k), torch.float32, 6)
    W = W.t() if w_t else W
    want = fx.linear(X, W)
    rest = [i for i in range(m) if i != 1]
    for bad in (float("inf"), float("-inf"), float("nan")):
        Y = X.clone()
        Y[1, 17] = bad
        got = fx.linear(Y, W, act="relu" if bad != float("-inf") else None)
        assert not torch.isfinite(got[1]).any()
        assert torch.equal(got[rest], want[rest])
        G = _positive((m, k), torch.float32, 7)
        base = fx.linear_grad(G, X, W)
        H = G.clone()
        H[1, 3] = bad
        dX, dW, db = fx.linear_grad(H, X, W)
        assert not torch.isfinite(dX[1]).any() and torch.equal(dX[rest], base[0][rest])
        cols = [j for j in range(k) if j != 3]
        assert not torch.isfinite(dW[:, 3]).any() and torch.equal(dW[:, cols], base[1][:, cols])
        assert not torch.isfinite(db[3]) and torch.equal(db[cols], base[2][cols])


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("m", [1, 5, 8, 16])
@pytest.mark.parametrize("pitch", [3, 4])
def test_few_rows_gradient_in_slices(m, pitch, w_t):
    """float32 gradients of few rows from column slices (poisoned around them) are those of whole tensors, to fp32 rounding: 2 u S sqrt(K) of
    two sums in orders of their own, 8 + 4 sqrt(K) taken."""
    n, k = 272, 200
    def cut(x):
        wide = torch.full((x.shape[0], x.shape[1] + pitch), float("nan"), device="cuda")
        wide[:, 1:1 + x.shape[1]] = x
        return wide[:, 1:1 + x.shape[1]]
    X, G, Z = (_positive(s, torch.float32, 8 + i) - 1.5 for i, s in enumerate([(m, n), (m, k), (m, k)]))
    W = _positive((k, n) if w_t else (n, k), torch.float32, 11) - 1.5
    turn = (lambda x: x.t()) if w_t else (lambda x: x)
    got = fx.linear_grad(cut(G), cut(X), turn(cut(W)), pre=cut(Z), act="silu")
    D = G.double() * torch.sigmoid(Z.double()) * (1 + Z.double() * torch.sigmoid(-Z.double()))
    A, B = X.double(), turn(W).double()
    for x, want, S, K in zip(got, (D @ B.t(), A.t() @ D, D.sum(0)),
                             (D.abs() @ B.abs().t(), A.abs().t() @ D.abs(), D.abs().sum(0)), (k, m, m)):
        # D itself to 32 u of its terms, as the slopes are
        assert ((x.double() - want).abs() <= (8 + 4 * K**0.5 + 32) * 2.0**-24 * S + 2.0**-24 * want.abs() + 2.0**-20 * (S == 0)).all()


@pytest.mark.parametrize("size", [1e-30, 1e-34, 1e-36, 1e-38])
@pytest.mark.parametrize("m,n,k", [(300, 200, 136), (300, 24, 40), (4, 200, 136)])
def test_tiny_float32_values(m, n, k, size):
    """float32 values so small that their terms end at bfloat16's smallest number, 2^-133: each is taken to within half of
    that, on top of the usual (8 + 4 sqrt(K)) u S."""
    X, W = (_positive(s, torch.float32, 12 + i) - 1.5 for i, s in enumerate([(m, n), (n, k)]))
    X = X * size
    got = fx.linear(X, W)
    x, w = X.double(), W.double()
    tol = (8 + 4 * n**0.5) * 2.0**-24 * (x.abs() @ w.abs()) + 2.0**-134 * w.abs().sum(0) + 2.0**-149
    assert ((got.double() - x @ w).abs() <= tol).all()


# Each way that a sum of more than 8,192 terms is laid over the tensor cores, entry by entry: narrow tiles by columns (16, 32 and
# 64 rows), single CTAs and pairs with one tile or many in turn, and sums split through a workspace, some of them not into
# equal pieces.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("shape", [(10, 70_000, 20_000), (30, 20_000, 40_000), (60, 20_000, 40_000), (100, 20_000, 40_000),
                                   (300, 20_000, 4096), (1000, 12_000, 4000), (5000, 8200, 5000), (40_000, 8300, 64),
                                   (40_000, 8300, 100), (20_000, 33_000, 200), (1, 9000, 100_000), (300, 8193, 9728)], ids=str)
def test_long_sums_entry_by_entry(shape, dtype):
    check_linear(*shape, dtype, act="silu", w_t=shape[0] % 3 == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("shape", [(20_000, 300, 520), (9000, 4096, 264), (70_000, 72, 1000)], ids=str)
def test_long_gradients_entry_by_entry(shape, dtype):
    check_grad(*shape, dtype, act="gelu", w_t=shape[0] == 9000)
