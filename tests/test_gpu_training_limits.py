"""Layer norm, the embedding lookup, cross entropy and their gradients where one of them was wrong or took too much: long logits of
terms of one sign, weights of rows that are left out, rows around a large mean, workspace, a classifier of no rows, a gain beside the weights."""
import math

import pytest
import torch

import dense_linear_algebra_gb300 as fx
from dense_linear_algebra_gb300 import solvers
from test_gpu_cross_entropy import check

pytestmark = pytest.mark.gpu

U = 2.0**-24
W_OF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [2048, 4096, 8192, 9000])
@pytest.mark.parametrize("m,k", [(200, 300), (40, 5000)])
def test_logits_of_terms_of_one_sign(m, k, n, dtype):
    """The gradient's logits are those of the loss: what the tensor cores cut off of them, 6.3e-9 of a sum of terms of one sign for
    each of at most 1,024 features, cancels in exp(z - lse).

    Every z is near S = 400, all of its terms positive. With lse in 64 bits z is short by between 0 and 6.5e-6 S and rounded once
    for each of the n / 1024 pieces, u S each; with the loss's own lse the shortfalls differ by as much at most, and those lse are off
    by that and by the sum's (8 + 4 sqrt(k)) u. exp(z - lse) adds 2 u S of its argument (the subtraction, lse's own rounding) and
    (2 |z - lse| + 8) u, db the sum's (8 + 4 sqrt(m)) u and the roundoff of its type (float16 also half its smallest number).
    """
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    X = (torch.rand(m, n, generator=gen, device="cuda") + 0.5).to(dtype)
    W = ((torch.rand(k, n, generator=gen, device="cuda") + 0.5) * (400 / n)).to(dtype).t()
    labels = torch.zeros(m, dtype=torch.int64, device="cuda")  # the other classes' db is a sum of probabilities
    z = X.double() @ W.double()
    lse = torch.logsumexp(z, 1)
    _, own = fx.cross_entropy(X, W, labels)
    S = float(z.max())
    dz = (6.5e-6 + (n // 1024 + 3) * U) * S
    d_lse = dz + (8 + 4 * k**0.5 + 40) * U + U * S
    assert float((own.double() - lse).abs().max()) <= d_lse
    p = torch.exp(z - lse[:, None])[:, 1:]
    want = p.sum(0)
    rel = (2 * (lse[:, None] - z)[:, 1:].abs().max() + 8) * U + 2 * U * S + (8 + 4 * m**0.5) * U
    for given, off in ((lse.float(), dz), (own, dz + (8 + 4 * k**0.5 + 40) * U)):
        db = fx.cross_entropy_grad(X, W, labels, given, need=(False, False, True))[2]
        err = ((db.double()[1:] - want) / want).abs()
        tol = (off + rel + W_OF[dtype]) * 1.01 + (2.0**-25 / want if dtype is torch.float16 else 0.0)
        assert bool((err <= tol).all()), float((err / tol).max())
    # with the loss's own lse a row's probabilities add up to one as fp32 sums do
    D = fx.cross_entropy_grad(X, W, labels, own, g=64.0, need=(False, False, True))[2].double()
    total = float(D.sum()) / 64
    slack = m * ((2 * float((lse[:, None] - z).max()) + 8 + 8 + 4 * k**0.5 + 40) * U + 2 * U * S) + W_OF[dtype] * float(D.abs().sum()) / 64
    assert abs(total) <= slack, (total, slack)


@pytest.mark.parametrize("m,n,k", [(200, 40, 20), (3, 100, 300), (200, 100, 300), (8193, 24, 10), (40_000, 72, 70)])
@pytest.mark.parametrize("weight", [1e20, float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_weights_of_rows_without_a_label(m, n, k, weight, dtype):
    """They have no say, in the power of two that float16's D is held at neither.

    db is D's sum: of each entry z and lse are off by at most 2.5e-5 (48 u S, S below 9), the exponential by 2e-6, the sum by 5e-5
    ((8 + 4 sqrt(m)) u): 1e-4 of the magnitudes' sum.
    """
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    X = torch.randn(m, n, generator=gen, device="cuda").to(dtype)
    W = (torch.randn(k, n, generator=gen, device="cuda") / n**0.5).to(dtype).t()
    labels = torch.randint(0, k, (m,), generator=gen, device="cuda")
    out = torch.arange(m, device="cuda") % 3 == 1
    labels[out] = torch.where(torch.arange(int(out.sum()), device="cuda") % 2 == 0, -1, k)
    _, lse = fx.cross_entropy(X, W, labels)
    # the largest weight stands in the last row that has a label, behind many others
    g = torch.full((m,), 1e-3, device="cuda")
    g[int((~out).nonzero()[-1])] = 3e-2
    g[out] = 0
    want = fx.cross_entropy_grad(X, W, labels, lse, g=g)
    g[out] = weight
    got = fx.cross_entropy_grad(X, W, labels, lse, g=g)
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(got, want))
    z = X.double() @ W.double()
    D = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    D[torch.arange(m, device="cuda"), torch.where(out, 0, labels)] -= 1
    D *= torch.where(out, 0.0, g.double())[:, None]
    tol = (W_OF[dtype] * D.sum(0).abs() + 1e-4 * D.abs().sum(0)) + (2.0**-25 if dtype is torch.float16 else 0)
    assert bool(((got[2].double() - D.sum(0)).abs() <= tol).all())
    # all rows left out: nothing
    none = fx.cross_entropy_grad(X, W, torch.full_like(labels, -1), lse, g=torch.full((m,), weight, device="cuda"))
    assert not any(t.any() for t in none)


# a register, a ring, a short, an odd and a long row's kernel, each with threads beyond the row's end
@pytest.mark.parametrize("m,n,dtype", [(9, 301, torch.float32), (9, 280, torch.bfloat16), (3100, 1160, torch.float32), (5000, 280, torch.bfloat16),
                                       (62_300, 20, torch.float32), (120_000, 24, torch.bfloat16), (5000, 301, torch.float32), (3001, 2047, torch.bfloat16),
                                       (5, 10_000, torch.float32), (5, 9001, torch.bfloat16)])
def test_norm_of_rows_around_a_large_mean(m, n, dtype):
    """mean rstd is beyond fp32 (1e39), x - mean is zero: u is zero, and dX = rstd (g - avg g) + r.

    avg g is off by C = 80 roundings of avg |g|, as in the norm's other tests, the rest by three of each term.
    """
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    X = torch.full((m, n), 1e36, device="cuda").to(dtype)
    G, R = (torch.randn(m, n, generator=gen, device="cuda").to(dtype) for _ in range(2))
    mean, rstd = X[:, 0].float().contiguous(), torch.full((m,), 1e3, device="cuda")
    dX, dw, db = fx.layer_norm_grad(G, X, None, mean, rstd, residual=R)
    g, r = G.double(), R.double()
    c = g.mean(1, keepdim=True)
    want = 1e3 * (g - c) + r
    tol = 1e3 * (80 * U * g.abs().mean(1, keepdim=True) + 4 * U * (g.abs() + c.abs())) + 2 * U * r.abs()
    err = (dX.double() - want).abs()
    assert bool((err <= tol + W_OF[dtype] * (want.abs() + tol)).all())
    assert not dw.any() and bool(((db.double() - g.sum(0)).abs() <= (8 + 4 * m**0.5) * U * g.abs().sum(0) + W_OF[dtype] * g.sum(0).abs() * 1.001).all())


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("m", [5, 9, 12, 16, 17, 128, 129])
def test_workspace_of_a_few_float32_rows(m, w_t, monkeypatch):
    """W's planes (600 MB for all classes) go in pieces of up to 512 MB whatever the rows' number; the other arrays of an allocation are
    below 64 MB."""
    monkeypatch.setenv("FXTX_FAIL_ALLOC_ABOVE", str(576_000_000))
    check(m, 1000, 100_001, torch.float32, w_t=w_t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [0, 50])
def test_a_classifier_of_no_rows(tokens, dtype):
    """Nothing to classify, and nothing to learn from."""
    X = torch.empty((0, 3), dtype=torch.int64, device="cuda") if tokens else torch.empty((0, 20), device="cuda")
    labels = torch.empty(0, dtype=torch.int64, device="cuda")
    net, info = solvers.classify_adamw(X, labels, 7, hidden=72, layers=1, tokens=tokens, width=16, steps=2, dtype=dtype)
    assert info.steps == 2 and not torch.stack(info.losses).any()
    fresh = solvers.Classifier(3 * 16 if tokens else 20, 72, 7, 1, tokens, 16, dtype=dtype)
    assert all(torch.equal(a, b) for a, b in zip(net.parameters(), fresh.parameters()))
    assert net.logits(X if tokens else X.to(dtype)).shape == (0, 7)


@pytest.mark.parametrize("k", range(1, 18))
@pytest.mark.parametrize("n", [3, 16, 24, 32, 61, 64])
def test_every_number_of_few_classes(n, k):
    """Float32 rows of few features and classes, whose kernels hold the classes in pairs; one row too few for those kernels too."""
    for m in (5000 * k - 1, 8000 * k + 1):
        check(m, n, k, torch.float32, bias=k % 2 == 0, w_t=n % 2 == 0, need=(k % 3 != 0, True, True))


@pytest.mark.parametrize("dtype,code", [(torch.float32, 0), (torch.bfloat16, 1), (torch.float16, 2)])
@pytest.mark.parametrize("m,n,k", [(200, 40, 20), (3, 100, 300), (200, 100, 300), (70_000, 32, 10)])
@pytest.mark.parametrize("gain", [1e-30, 2.0**120])
def test_a_gain_beside_the_weights(m, n, k, gain, dtype, code):
    """gain G is what counts, whatever the size of each: a power of two in one and its inverse in the other changes no bit."""
    gain = 2.0 ** round(math.log2(gain))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    X = torch.randn(m, n, generator=gen, device="cuda").to(dtype)
    P = (torch.randn(k, n, generator=gen, device="cuda") / n**0.5).to(dtype)
    labels = torch.randint(-1, k, (m,), generator=gen, device="cuda")
    g = torch.rand(m, generator=gen, device="cuda") + 0.5
    _, lse = fx.cross_entropy(X, P.t(), labels)
    want = fx.cross_entropy_grad(X, P.t(), labels, lse, g=g)
    dX, dP, db = torch.empty_like(X), torch.empty_like(P), torch.empty(k, dtype=dtype, device="cuda")
    weights = g / gain
    rc = fx.fxtx_cross_entropy_grad(code, m, n, k, X.data_ptr(), n, P.data_ptr(), n, 1, None, labels.data_ptr(), 64, lse.data_ptr(),
                                    weights.data_ptr(), gain, dX.data_ptr(), n, dP.data_ptr(), n, db.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream)
    assert rc == fx.FXTX_OK
    assert torch.equal(dX, want[0]) and torch.equal(dP.t(), want[1]) and torch.equal(db, want[2])
