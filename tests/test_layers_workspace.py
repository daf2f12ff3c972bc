"""Workspace of the layer calls."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(code, **env):
    run = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, env=dict(os.environ, **env), timeout=300,
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-2000:]


@pytest.mark.gpu
def test_a_pool_that_could_not_be_made_is_tried_again():
    """FXTX_FAIL_POOL makes the pool's creation fail, as a lack of memory would: that call reports it, the next one has its pool."""
    _child("""
        import os
        import torch
        import dense_linear_algebra_gb300 as fx
        X, W = torch.randn(300, 200, device="cuda"), torch.randn(200, 136, device="cuda")
        os.environ["FXTX_FAIL_POOL"] = "1"
        try:
            fx.linear(X, W)
        except fx.FxtxError as e:
            assert e.status == fx.FXTX_ERR_ALLOC
        else:
            raise SystemExit("the call did not report its failure")
        del os.environ["FXTX_FAIL_POOL"]
        assert float((fx.linear(X, W) - X @ W).abs().max()) < 0.1
    """)


@pytest.mark.gpu
def test_first_call_in_a_capture():
    """The first layer call of a process may be one that a graph captures."""
    _child("""
        import torch
        import dense_linear_algebra_gb300 as fx
        torch.manual_seed(0)
        X, W = torch.randn(300, 200, device="cuda"), torch.randn(200, 136, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fx.linear(X, W)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, fx.linear(X, W))
        assert float((got - X @ W).abs().max()) < 0.1
    """)
