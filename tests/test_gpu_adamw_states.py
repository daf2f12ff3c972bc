"""AdamW's held states where they go wrong quietly: blocks that are not finite."""
import pytest
import torch

import dense_linear_algebra_gb300 as fx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3e38, -1e25])
def test_8_bit_second_moment_of_a_block_that_is_not_finite(bad):
    """Where a gradient is not finite, or its square is not, the block's second moments are NaN, those of elements whose gradient was zero among
    them, and so are its params from the next step on; the other blocks go on as they would."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    p, g = (torch.randn(1000, generator=gen, device="cuda") for _ in range(2))
    g[260:270] = 0
    q, clean = p.clone(), g.clone()
    g[300] = bad
    a, b = fx.AdamW([p], state_bits=8, lr=1e-2), fx.AdamW([q], state_bits=8, lr=1e-2)
    block = torch.zeros(1000, dtype=torch.bool, device="cuda")
    block[256:512] = True
    for step in range(2):
        a.step([g if step == 0 else clean])
        b.step([clean])
        (m, v), (n, w) = a.moments(), b.moments()
        assert torch.isnan(v[:1000][block]).all() and torch.equal(v[:1000][~block], w[:1000][~block])
        assert torch.equal(m[:1000][~block], n[:1000][~block])
        if not abs(bad) < float("inf"):
            assert torch.isnan(m[:1000][block]).all()
    assert torch.isnan(p[block]).all() and torch.equal(p[~block], q[~block])
