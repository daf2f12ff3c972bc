"""The training operators together: a classifier on features or ids (solvers.Classifier, solvers.classify_adamw)."""
import pytest
import torch

from dense_linear_algebra_gb300 import solvers

pytestmark = pytest.mark.gpu


def problem(m, classes, tokens, slots, n, dtype, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if tokens:
        X = torch.randint(-1, tokens, (m, slots), generator=gen, device="cuda")  # -1: padding
    else:
        X = torch.randn(m, n, generator=gen, device="cuda").to(dtype)
    labels = torch.randint(-1, classes + 1, (m,), generator=gen, device="cuda")  # -1, classes: left out
    return X, labels


def net64(net, X, labels):
    """The mean loss and its gradients in 64 bits, by torch's autograd on the working parameters."""
    p = {name: w.detach().double().requires_grad_(True) for name, w in net.working().items()}
    if net.tokens:
        inside = (X >= 0) & (X < net.tokens)
        x = torch.where(inside[..., None], p["table"][torch.where(inside, X, 0)], 0.0) * net.width**0.5
        x = x.reshape(X.shape[0], -1)
    else:
        x = X.double()
    v, h = x, 0.0
    for i in range(net.layers + 1):
        z = v @ p[f"W{i}"] + p[f"b{i}"]
        h = h + z * torch.special.ndtr(z)
        v = torch.nn.functional.layer_norm(h, (h.shape[1],), p[f"g{i}"], p[f"s{i}"], 1e-5)
    logits = v @ p["P"].t() + p["c"]
    y = torch.where((labels >= 0) & (labels < logits.shape[1]), labels, -100)
    loss = torch.nn.functional.cross_entropy(logits, y, ignore_index=-100)
    return logits, loss, torch.autograd.grad(loss, list(p.values()))


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-5), (torch.bfloat16, 0.08), (torch.float16, 0.015)])
@pytest.mark.parametrize("m,classes,hidden,layers,tokens,slots,n", [
    (300, 10, 96, 2, 0, 0, 40),      # a layer of tensor-core tiles, few classes
    (1000, 12, 48, 1, 0, 0, 32),     # thin layers throughout
    (257, 700, 72, 1, 90, 3, 0),     # ids, many classes
    (9, 130, 80, 0, 50, 2, 0),       # few rows
])
def test_gradients_against_autograd(m, classes, hidden, layers, tokens, slots, n, dtype, tol):
    """All parameters' gradients: relative to their size, the roundings to the type of each layer's result, norm, D and gradient (at
    most five a layer, each its unit roundoff, through at most three layers, the classes and the table), for float32 fp32 sums."""
    X, labels = problem(m, classes, tokens, slots, n, dtype)
    net = solvers.Classifier(n or slots * 24, hidden, classes, layers, tokens, 24, "gelu", dtype)
    logits, loss, want = net64(net, X, labels)
    got, kept = net.loss(X, labels)
    inside = (labels >= 0) & (labels < classes)
    assert not got[~inside].any()
    loss = float(loss.detach())
    assert abs(float(got.double().sum() / inside.sum()) - loss) <= tol * abs(loss)
    assert float((net.logits(X).double() - logits.detach()).norm() / logits.detach().norm()) <= tol
    grads = solvers._mean_loss_gradients(net, labels, kept)
    for name, a, b in zip(net.params, grads, want):
        assert a.shape == b.shape, name
        assert float((a.double() - b).norm() / b.norm().clamp_min(1e-30)) <= tol, name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [0, 60])
def test_training_runs_and_repeats(tokens, dtype):
    """Short last batches, padding and rows without a label; the same parameters bit for bit on every run."""
    X, labels = problem(1000, 30, tokens, 4, 20, torch.float32)
    runs = [solvers.classify_adamw(X, labels, 30, hidden=80, layers=1, tokens=tokens, width=16, steps=6, batch=384, state_bits=8,
                                   dtype=dtype) for _ in range(2)]
    (a, info), (b, _) = runs
    assert info.steps == 6 and torch.isfinite(torch.stack(info.losses)).all()
    for x, y in zip(a.parameters(), b.parameters()):
        assert torch.equal(x, y) and torch.isfinite(x).all()


def test_rows_without_a_label_have_no_say():
    """A batch with rows left out gives the gradients of the batch without them."""
    X, labels = problem(400, 25, 0, 0, 30, torch.float32)
    inside = (labels >= 0) & (labels < 25)
    net = solvers.Classifier(30, 72, 25)
    a = solvers._mean_loss_gradients(net, labels, net.loss(X, labels)[1])
    b = solvers._mean_loss_gradients(net, labels[inside], net.loss(X[inside], labels[inside])[1])
    for x, y in zip(a, b):
        # sums of the same terms in another order, over at most 400 rows
        assert float((x - y).norm() / y.norm()) <= 400**0.5 * 2.0**-22
