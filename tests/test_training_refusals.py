"""What layer norm, the embedding lookup, cross entropy and their gradients refuse, before anything reaches a device: in the C entries
and in the binding."""
import pytest
import torch

import dense_linear_algebra_gb300 as fx

BAD = fx.FXTX_ERR_INVALID_ARG
P = 4096  # stands for a pointer; nothing here gets as far as reading it


def test_layer_norm_entries():
    ok = [0, 4, 8, P, 8, None, None, 1e-5, P, 8, None, None, None]
    norm = lambda **k: fx.fxtx_layer_norm(*[k.get(f"a{i}", v) for i, v in enumerate(ok)])  # noqa: E731
    assert norm(a0=3) == BAD and norm(a0=-1) == BAD  # type
    assert norm(a1=-1) == BAD and norm(a2=-1) == BAD and norm(a2=0) == BAD and norm(a1=2**31) == BAD
    assert norm(a3=None) == BAD and norm(a8=None) == BAD
    assert norm(a4=7) == BAD and norm(a9=7) == BAD
    assert norm(a7=-1e-9) == BAD and norm(a7=float("nan")) == BAD and norm(a7=float("inf")) == BAD
    assert norm(a1=0, a3=None, a8=None) == fx.FXTX_OK

    ok2 = [1, 4, 8, P, 8, P, 8, None, P, P, None, 0, P, 8, P, P, None]
    grad = lambda **k: fx.fxtx_layer_norm_grad(*[k.get(f"a{i}", v) for i, v in enumerate(ok2)])  # noqa: E731
    assert grad(a0=7) == BAD and grad(a1=-1) == BAD and grad(a2=0) == BAD
    assert grad(a3=None) == BAD and grad(a5=None) == BAD and grad(a8=None) == BAD and grad(a9=None) == BAD
    assert grad(a4=7) == BAD and grad(a6=7) == BAD and grad(a13=7) == BAD and grad(a10=P, a11=7) == BAD
    assert grad(a12=None, a14=None, a15=None) == fx.FXTX_OK  # nothing wanted


def test_embedding_entries():
    ok = [0, 4, 8, 10, P, 64, P, 8, 1.0, P, 8, None]
    look = lambda **k: fx.fxtx_embedding(*[k.get(f"a{i}", v) for i, v in enumerate(ok)])  # noqa: E731
    assert look(a0=3) == BAD and look(a1=-1) == BAD and look(a2=-1) == BAD and look(a3=-1) == BAD and look(a3=2**31) == BAD
    assert look(a4=None) == BAD and look(a5=16) == BAD and look(a6=None) == BAD and look(a7=7) == BAD
    assert look(a9=None) == BAD and look(a10=7) == BAD
    assert look(a1=0, a4=None, a9=None) == fx.FXTX_OK and look(a2=0, a6=None, a9=None) == fx.FXTX_OK

    ok2 = [0, 4, 8, 10, P, 8, P, 32, 1.0, P, 8, None]
    grad = lambda **k: fx.fxtx_embedding_grad(*[k.get(f"a{i}", v) for i, v in enumerate(ok2)])  # noqa: E731
    assert grad(a0=3) == BAD and grad(a1=-1) == BAD and grad(a2=-1) == BAD and grad(a3=-1) == BAD
    assert grad(a4=None) == BAD and grad(a5=7) == BAD and grad(a6=None) == BAD and grad(a7=0) == BAD
    assert grad(a9=None) == BAD and grad(a10=7) == BAD
    assert grad(a3=0, a9=None) == fx.FXTX_OK and grad(a2=0, a4=None, a9=None) == fx.FXTX_OK


def test_cross_entropy_entries():
    ok = [0, 4, 8, 10, P, 8, P, 8, 1, None, P, 64, P, P, None]
    loss = lambda **k: fx.fxtx_cross_entropy(*[k.get(f"a{i}", v) for i, v in enumerate(ok)])  # noqa: E731
    assert loss(a0=3) == BAD and loss(a1=-1) == BAD and loss(a2=0) == BAD and loss(a3=0) == BAD and loss(a3=2**31) == BAD
    assert loss(a4=None) == BAD and loss(a5=7) == BAD and loss(a6=None) == BAD and loss(a7=7) == BAD and loss(a8=2) == BAD
    assert loss(a8=0, a7=9) == BAD and loss(a10=None) == BAD and loss(a11=8) == BAD
    assert loss(a1=0, a4=None, a10=None) == fx.FXTX_OK and loss(a12=None, a13=None) == fx.FXTX_OK

    ok2 = [0, 4, 8, 10, P, 8, P, 8, 1, None, P, 64, P, None, 1.0, P, 8, P, 8, P, None]
    grad = lambda **k: fx.fxtx_cross_entropy_grad(*[k.get(f"a{i}", v) for i, v in enumerate(ok2)])  # noqa: E731
    assert grad(a0=3) == BAD and grad(a1=-1) == BAD and grad(a2=0) == BAD and grad(a3=0) == BAD
    assert grad(a4=None) == BAD and grad(a5=7) == BAD and grad(a6=None) == BAD and grad(a7=7) == BAD and grad(a8=2) == BAD
    assert grad(a10=None) == BAD and grad(a11=8) == BAD and grad(a12=None) == BAD
    assert grad(a16=7) == BAD and grad(a18=7) == BAD and grad(a8=0, a7=10, a18=9) == BAD
    assert grad(a15=None, a17=None, a19=None) == fx.FXTX_OK


def test_host_tensors():
    X, v = torch.zeros(8, 4), torch.zeros(8)
    ids = torch.zeros(8, dtype=torch.int64)
    for call in (lambda: fx.layer_norm(X), lambda: fx.layer_norm_grad(X, X, None, v, v), lambda: fx.embedding(ids, X),
                 lambda: fx.embedding_grad(X, ids, 4), lambda: fx.cross_entropy(X, X.t(), ids),
                 lambda: fx.cross_entropy_grad(X, X.t(), ids, v)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding():
    X, v = torch.zeros((8, 4), device="cuda"), torch.zeros(8, device="cuda")
    ids, W = torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros((4, 5), device="cuda")
    bad = [
        (ValueError, lambda: fx.layer_norm(X.t())), (ValueError, lambda: fx.layer_norm(X, v)),
        (ValueError, lambda: fx.layer_norm(X, v[:4].double())), (ValueError, lambda: fx.layer_norm(X, out=X[:4])),
        (TypeError, lambda: fx.layer_norm(X.double())), (ValueError, lambda: fx.layer_norm(X[0])),
        (ValueError, lambda: fx.layer_norm_grad(X[:4], X, None, v, v)), (ValueError, lambda: fx.layer_norm_grad(X, X, None, v[:4], v)),
        (ValueError, lambda: fx.layer_norm_grad(X, X, None, None, None)), (ValueError, lambda: fx.layer_norm_grad(X, X, None, v.half(), v)),
        (ValueError, lambda: fx.layer_norm_grad(X, X, None, v, v, residual=X.bfloat16())),
        (TypeError, lambda: fx.embedding(v, X)), (ValueError, lambda: fx.embedding(ids.view(2, 4), X)),
        (ValueError, lambda: fx.embedding(ids.cpu(), X)), (ValueError, lambda: fx.embedding(ids[::2], X)),
        (ValueError, lambda: fx.embedding(ids, X.t())), (ValueError, lambda: fx.embedding(ids, X, out=X[:4])),
        (ValueError, lambda: fx.embedding_grad(X, ids[:4], 3)), (ValueError, lambda: fx.embedding_grad(X, ids, -1)),
        (ValueError, lambda: fx.embedding_grad(X, ids, 3, out=X)), (TypeError, lambda: fx.embedding_grad(X, ids.short(), 3)),
        (ValueError, lambda: fx.cross_entropy(X, W[:3], ids)), (ValueError, lambda: fx.cross_entropy(X, W, ids[:4])),
        (TypeError, lambda: fx.cross_entropy(X, W, v)), (ValueError, lambda: fx.cross_entropy(X, W, ids, v)),
        (ValueError, lambda: fx.cross_entropy(X, W.bfloat16(), ids)), (TypeError, lambda: fx.cross_entropy(X.double(), W, ids)),
        (ValueError, lambda: fx.cross_entropy_grad(X, W, ids, v[:4])), (ValueError, lambda: fx.cross_entropy_grad(X, W, ids, None)),
        (ValueError, lambda: fx.cross_entropy_grad(X, W, ids, v.half())), (ValueError, lambda: fx.cross_entropy_grad(X, W, ids, v, g=v[:4])),
        (ValueError, lambda: fx.cross_entropy_grad(X, W, ids, v, g=v.half())), (fx.FxtxError, lambda: fx.cross_entropy(X, W[:, :0], ids)),
        (fx.FxtxError, lambda: fx.cross_entropy(X[:, :0], W[:0], ids)), (fx.FxtxError, lambda: fx.layer_norm(X[:, :0])), (fx.FxtxError, lambda: fx.layer_norm(X, eps=-1.0)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
