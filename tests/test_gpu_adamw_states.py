"""AdamW's held states where they go wrong quietly: blocks that are not finite, and states of other tensors."""
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


@pytest.mark.parametrize("bits", [8, 32])
def test_states_of_other_tensors_are_refused(bits):
    """The same number of elements in other tensors, in all or block by block, is not the same state; a state without its step count
    is refused before anything is taken from it."""
    def made(sizes):
        return fx.AdamW([torch.zeros(n, device="cuda") for n in sizes], state_bits=bits)

    a = made([256, 512])
    a.step([torch.ones(256, device="cuda"), torch.ones(512, device="cuda")])
    saved = a.state_dict()
    for sizes in ([512, 256], [768], [255, 512], [256, 512, 0]):
        b = made(sizes)
        with pytest.raises(ValueError):
            b.load_state_dict(saved)
        assert b.steps == 0 and not b.exp_avg.any()
    b = made([256, 512])
    with pytest.raises(ValueError):
        b.load_state_dict({k: v for k, v in saved.items() if k != "steps"})
    assert b.steps == 0 and not b.exp_avg.any()
    b.load_state_dict(saved)
    assert b.steps == 1 and torch.equal(b.exp_avg, a.exp_avg)
    # a state put together by hand may leave the sizes out
    c = made([256, 512])
    c.load_state_dict({k: v for k, v in saved.items() if k != "sizes"})
    assert c.steps == 1 and torch.equal(c.exp_avg_sq, a.exp_avg_sq)
