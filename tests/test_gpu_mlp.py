"""The layer operators together: a residual network trained with AdamW (solvers.mlp_adamw)."""
import pytest
import torch

from dense_linear_algebra_gb300 import solvers

pytestmark = pytest.mark.gpu


def _problem(m, n, k, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    X = torch.randn(m, n, generator=gen, device="cuda")
    A, C = torch.randn(n, 16, generator=gen, device="cuda") / n ** 0.5, torch.randn(16, k, generator=gen, device="cuda") / 4
    return X, torch.tanh(2 * X @ A) @ C


def _net64(net, X):
    """The network and its gradient in 64 bits, by torch's autograd on the working weights."""
    W, b = net._working()
    W, b = [w.double().requires_grad_(True) for w in W], [x.double().requires_grad_(True) for x in b]
    h = X.double()
    for i in range(len(W)):
        z = h @ W[i] + b[i]
        if i == len(W) - 1:
            return z, W + b
        a = z * torch.special.ndtr(z)
        h = h + a if i else a


@pytest.mark.parametrize("layers", [0, 1, 3])
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 0.05), (torch.float16, 0.01)])
def test_network_gradient_against_autograd(layers, dtype, tol):
    """Gradients of all layers against autograd in 64 bits: relative to their size, the roundings to the type of each
    layer's result, D and gradient (at most three a layer, each its unit roundoff, over at most five layers) and
    for float32 fp32 sums."""
    X, _ = _problem(300, 40, 8)
    X = X.to(dtype)
    net = solvers.MLP(40, 96, 8, layers, "gelu", dtype)
    G = torch.randn(300, 8, device="cuda").to(dtype)
    out, saved = net.forward(X, keep=True)
    assert torch.equal(out, net.forward(X))
    want, params = _net64(net, X)
    assert float((out.double() - want.detach()).norm() / want.detach().norm()) <= tol
    grads = torch.autograd.grad(want, params, G.double())
    for got, ref in zip(net.backward(G, saved), grads):
        assert got.shape == ref.shape
        assert float((got.double() - ref).norm() / ref.norm()) <= tol


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("state_bits", [32, 8])
def test_training_learns(dtype, state_bits):
    """The loss of a function that the network can represent falls to a tenth in 300 steps."""
    X, B = _problem(4096, 32, 4)
    net, info = solvers.mlp_adamw(X, B, hidden=128, layers=2, steps=300, batch=1024, lr=3e-3, state_bits=state_bits,
                                  dtype=dtype)
    first, last = float(info.losses[0]), float(torch.stack(info.losses[-20:]).mean())
    assert info.steps == 300 and last < 0.1 * first
    assert float((net.forward(X.to(dtype)).float() - B).square().mean()) < 0.15 * first


def test_training_repeats_bit_by_bit():
    X, B = _problem(1000, 20, 3)
    a, _ = solvers.mlp_adamw(X, B, hidden=80, layers=1, steps=5, batch=256, state_bits=8, dtype=torch.bfloat16)
    b, _ = solvers.mlp_adamw(X, B, hidden=80, layers=1, steps=5, batch=256, state_bits=8, dtype=torch.bfloat16)
    for x, y in zip(a.parameters() + a.copies, b.parameters() + b.copies):
        assert torch.equal(x, y)
