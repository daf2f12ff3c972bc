"""mlp_adamw: every row is trained on, whatever the batch, and float16 trains on as many rows as float32 does."""
import pytest
import torch

from dense_linear_algebra_gb300 import solvers
from dense_linear_algebra_gb300.layers import AdamW

pytestmark = pytest.mark.gpu


def _problem(m, n, k, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    X = torch.randn(m, n, generator=gen, device="cuda")
    return X, torch.tanh(X @ torch.randn(n, k, generator=gen, device="cuda") / n**0.5)


@pytest.mark.parametrize("m,batch", [(100, 64), (1000, 300), (64, 64), (7, 3)])
def test_batches_cover_all_rows(m, batch):
    """Two passes are the steps of a plain loop over slices of the rows, the last one short."""
    X, B = _problem(m, 12, 3)
    steps = 2 * -(-m // batch)
    net, info = solvers.mlp_adamw(X, B, hidden=70, layers=1, steps=steps, batch=batch)
    ref = solvers.MLP(12, 70, 3, 1, seed=0)
    opt = AdamW(ref.parameters(), lr=1e-3, weight_decay=0.0)
    losses = []
    for i in list(range(0, m, batch)) * 2:
        out, saved = ref.forward(X[i:i + batch], keep=True)
        err = out - B[i:i + batch]
        losses.append(err.square().mean())
        opt.step(ref.backward(err * (2.0 / err.numel()), saved))
    assert len(info.losses) == steps and torch.equal(torch.stack(info.losses), torch.stack(losses))
    for x, y in zip(net.parameters(), ref.parameters()):
        assert torch.equal(x, y)


def test_float16_learns_from_many_rows():
    """The gradient of a mean over millions of entries lies below float16's smallest numbers: it has to reach the weights all the
    same. float16's own roundings cost little: its loss ends within half of float32's, which has fallen to a hundredth."""
    X, B = _problem(8_000_000, 16, 4)
    loss = {}
    for dtype in (torch.float32, torch.float16):
        _, info = solvers.mlp_adamw(X, B, hidden=64, layers=1, steps=300, lr=3e-3, dtype=dtype)
        loss[dtype] = [float(info.losses[0]), float(info.losses[-1])]
    first, last = loss[torch.float32]
    assert last < 0.01 * first
    assert loss[torch.float16][1] <= 1.5 * last


@pytest.mark.parametrize("size", [1e-4, 1.0, 300.0])
def test_float16_takes_targets_of_any_size(size):
    """Small and large residuals alike: nothing overflows, and the loss falls."""
    X, B = _problem(5000, 16, 4, 1)
    _, info = solvers.mlp_adamw(X, B * size, hidden=64, layers=1, steps=40, lr=1e-3, dtype=torch.float16)
    losses = torch.stack(info.losses)
    assert torch.isfinite(losses).all() and losses[-1] < losses[0]
