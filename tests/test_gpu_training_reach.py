"""Layer norm, the embedding lookup, cross entropy and their gradients on the kernels that large and odd sizes take: in place, rows
that are not finite, long runs of one id, ids of 28 bits, few rows against many classes and features, calls without workspace, offsets beyond 32 bits."""
import pytest
import torch

import dense_linear_algebra_gb300 as fx
from test_gpu_cross_entropy import check
from test_gpu_embedding import check_gradient, ids_of
from test_gpu_norm import make
from test_gpu_training_workspace import inputs

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

# rings of whole rows, rings of odd widths, tiles of short rows, two passes
NORMS = [(6000, 2056), (4900, 700), (3001, 2047), (8001, 301), (100_003, 64), (100_001, 40), (40, 40_000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", NORMS)
def test_norm_in_place(m, n, dtype):
    """OUT over X; DX over each of G, X and R, with the column sums wanted too."""
    X, G, R = (make((m, n), dtype, s) for s in (1, 2, 3))
    w, b = make((1, n), dtype, 4)[0], make((1, n), dtype, 5)[0]
    want, mean, rstd = fx.layer_norm(X, w, b, stats=True)
    Y = X.clone()
    out, mean2, rstd2 = fx.layer_norm(Y, w, b, stats=True, out=Y)
    assert out is Y and torch.equal(Y, want) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    grads = fx.layer_norm_grad(G, X, w, mean, rstd, residual=R)
    for i in range(3):
        a = [G.clone(), X.clone(), R.clone()]
        dw, db = torch.empty(n, dtype=dtype, device="cuda"), torch.empty(n, dtype=dtype, device="cuda")
        rc = fx.fxtx_layer_norm_grad(CODE[dtype], m, n, a[0].data_ptr(), n, a[1].data_ptr(), n, w.data_ptr(), mean.data_ptr(),
                                     rstd.data_ptr(), a[2].data_ptr(), n, a[i].data_ptr(), n, dw.data_ptr(), db.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream)
        assert rc == fx.FXTX_OK
        assert all(torch.equal(p, q) for p, q in zip((a[i], dw, db), grads))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", NORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_of_rows_that_are_not_finite(m, n, bad, dtype):
    """The first, the last and one between come out as NaN and leave the others alone."""
    rows = [0, m // 2 + 1, m - 1]
    X, G = make((m, n), dtype, 1), make((m, n), dtype, 2)
    want, mean, rstd = fx.layer_norm(X, stats=True)
    dX, _, db = fx.layer_norm_grad(G, X, None, mean, rstd)
    Y = X.clone()
    Y[rows, n - 1] = bad
    out, mean, rstd = fx.layer_norm(Y, stats=True)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(out[keep], want[keep]) and torch.isnan(out[rows, n - 1]).all()
    got, dw, db2 = fx.layer_norm_grad(G, Y, None, mean, rstd)
    assert torch.equal(got[keep], dX[keep]) and torch.isnan(got[rows]).all() and torch.isnan(dw).all()
    assert torch.equal(db, db2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["one", "frequent", "padded", "sorted"])
def test_long_runs_of_wide_rows(kind, dtype):
    """Runs over many chunks where rows come by bulk copies (the last of them a part of a kilobyte)."""
    check_gradient(ids_of(kind, 5000, 300, 3), 300, 1032, dtype, scale=2.0)
    check_gradient(ids_of(kind, 700, 3, 4), 3, 4096, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["uniform", "frequent", "padded"])
def test_many_rows_of_odd_widths(kind, dtype):
    """Four entries a thread: chunks times entries beyond 1.2 million."""
    check_gradient(ids_of(kind, 8200, 3000, 5), 3000, 5001, dtype, scale=0.5)


@pytest.mark.parametrize("m", [5, 12_000, 66_000])
def test_a_table_of_28_bits(m):
    """Four passes, in both sorts."""
    count = 2**27
    ids = ids_of("uniform", m, count, 7)
    ids[:4] = torch.tensor([0, count - 1, count, -1], device="cuda")
    G = make((m, 1), torch.float32, 1)
    got = fx.embedding_grad(G, ids, count)
    want = torch.zeros((count, 1), device="cuda")
    inside = (ids >= 0) & (ids < count)
    want.index_add_(0, ids[inside], G[inside])
    once = torch.bincount(ids[inside], minlength=1) < 2 if m < 100 else None
    # a row of one term is that term; of c terms the two orders differ by c u of their magnitudes' sum at most, c below 8 here
    S = torch.zeros((count, 1), device="cuda").index_add_(0, ids[inside], G[inside].abs())
    assert bool(((got - want).abs() <= 16 * 2.0**-24 * S).all()) and (once is None or torch.equal(got, want))
    E = torch.arange(count, dtype=torch.float32, device="cuda").view(-1, 1)
    rows = fx.embedding(ids, E)
    assert torch.equal(rows[:, 0], torch.where(inside, ids, 0).float())


@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(1, 512, 131_072), (4, 520, 70_000), (4, 4096, 3000), (2, 2056, 32_000), (1, 9000, 500), (16, 4096, 2000)])
def test_few_rows_of_many_classes(m, n, k, dtype, w_t):
    """Sums of several parts, joined: the logits' and dX's."""
    check(m, n, k, dtype, w_t=w_t)


# of each size: whether layer_norm_grad, embedding_grad, cross_entropy and its gradient take workspace
SIZES = [((300, 200, 700, torch.bfloat16), (True, True, True, True)), ((9, 96, 130, torch.float32), (False, True, True, True)),
         ((3000, 32, 10, torch.float32), (True, True, False, True)), ((2000, 40, 50, torch.float16), (True, True, False, True)),
         ((20_000, 72, 300, torch.float16), (True, True, True, True)), ((40, 2056, 1000, torch.float32), (True, True, True, True)),
         ((100_000, 16, 4, torch.float32), (True, True, False, True)), ((3, 128, 900, torch.bfloat16), (False, True, True, True))]


@pytest.mark.parametrize("size,takes", SIZES)
def test_which_calls_take_workspace(size, takes, monkeypatch):
    """A call that does fails without, a call that does not gives its results."""
    s = inputs(*size, 1)
    k = size[2]
    _, mean, rstd = fx.layer_norm(s["X"], stats=True)
    _, lse = fx.cross_entropy(s["X"], s["W"], s["ids"], s["b"])
    calls = [lambda: fx.layer_norm_grad(s["G"], s["X"], None, mean, rstd), lambda: (fx.embedding_grad(s["G"], s["ids"], k),),
             lambda: fx.cross_entropy(s["X"], s["W"], s["ids"], s["b"]),
             lambda: fx.cross_entropy_grad(s["X"], s["W"], s["ids"], lse, s["b"])]
    for call, fails in zip(calls, takes):
        want = call()
        monkeypatch.setenv("FXTX_FAIL_ALLOC", "1")
        if fails:
            with pytest.raises(fx.FxtxError) as e:
                call()
            assert e.value.status == fx.FXTX_ERR_ALLOC
        else:
            assert all(torch.equal(a, b) for a, b in zip(call(), want))
        monkeypatch.delenv("FXTX_FAIL_ALLOC")
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.fixture
def wide():
    """A matrix of 2.4 billion entries: offsets beyond 32 bits."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    yield torch.randn(300_000, 8192, generator=gen, dtype=torch.bfloat16, device="cuda")
    torch.cuda.empty_cache()


def test_norm_beyond_32_bits(wide):
    """Rows at the end as a call on them alone has them. The kernels differ, so fp32 results do by at most 1e-6 of a row's entries
    (below 6); rounded to bfloat16, half a step each, two such results are up to one step of bfloat16 apart: 2^-7 of their size.
    """
    end = wide[-50:].clone()
    want, mean, rstd = fx.layer_norm(end, stats=True)
    got, mean2, rstd2 = fx.layer_norm(wide, stats=True)
    G = torch.full((50, 8192), 0.5, dtype=torch.bfloat16, device="cuda") + end
    grad = fx.layer_norm_grad(G, end, None, mean, rstd, need=(True, False, False))[0]
    for a, b in ((got[-50:], want), (mean2[-50:], mean), (rstd2[-50:], rstd)):
        assert bool(((a.double() - b.double()).abs() <= 2.0**-7 * b.double().abs() + 1e-6).all())
    del got
    G2 = wide.clone()
    G2[-50:] = G
    dX = fx.layer_norm_grad(G2, wide, None, mean2, rstd2, need=(True, False, False))[0]
    assert bool(((dX[-50:].double() - grad.double()).abs() <= 2.0**-7 * grad.double().abs() + 2e-6).all())


def test_lookup_beyond_32_bits(wide):
    ids = torch.tensor([299_999, 0, 262_143, 299_999, -1], device="cuda")
    rows = fx.embedding(ids, wide)
    assert torch.equal(rows[:4], wide[ids[:4]]) and not rows[4].any()
    ids = torch.full((300_000,), -1, device="cuda")
    ids[-3:] = torch.tensor([7, 5, 7], device="cuda")
    dE = fx.embedding_grad(wide, ids, 9)
    assert torch.equal(dE[5], wide[-2]) and torch.equal(dE[7], (wide[-3].float() + wide[-1].float()).bfloat16())
    assert not dE[:5].any() and not dE[6].any() and not dE[8:].any()
    G = wide[:3].clone()
    dE = fx.embedding_grad(G, torch.tensor([299_999, 1, 299_998], device="cuda"), 300_000, out=wide)
    assert dE is wide and torch.equal(dE[[299_999, 1, 299_998]], G) and not dE[2:299_998].any() and not dE[0].any()


def test_loss_beyond_32_bits(wide):
    """The last rows' losses and gradients as calls on them alone have them, within the roundings of z (n = 8192: its sums are those of
    tiles in both) and of bfloat16."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    W = (torch.randn(70, 8192, generator=gen, device="cuda") / 90).bfloat16().t()
    labels = torch.randint(-1, 71, (300_000,), generator=gen, device="cuda")
    loss, lse = fx.cross_entropy(wide, W, labels)
    want, lse_end = fx.cross_entropy(wide[-200:], W, labels[-200:])
    assert bool(((loss[-200:] - want).abs() <= 1e-5).all()) and bool(((lse[-200:] - lse_end).abs() <= 1e-5).all())
    dX, _, _ = fx.cross_entropy_grad(wide, W, labels, lse, need=(True, False, False))
    end, _, _ = fx.cross_entropy_grad(wide[-200:], W, labels[-200:], lse_end, need=(True, False, False))
    assert float((dX[-200:].double() - end.double()).norm()) <= 2.0**-7 * float(end.double().norm())
