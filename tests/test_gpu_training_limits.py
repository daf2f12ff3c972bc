"""Layer norm, the embedding lookup, cross entropy and their gradients where one of them was wrong or took too much: long logits of
terms of one sign."""
import pytest
import torch

import dense_linear_algebra_gb300 as fx

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
