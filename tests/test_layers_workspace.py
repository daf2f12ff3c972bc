"""Workspace of the layer calls: a pool that could not be made is tried again, a first call may be captured, and memory that
torch holds on to is given back before a call fails."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import dense_linear_algebra_gb300 as fx
from dense_linear_algebra_gb300 import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(code, **env):
    run = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, env=dict(os.environ, **env), timeout=300,
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-2000:]


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


@pytest.mark.parametrize("capturing", [False, True])
def test_cached_memory_is_given_back_before_a_call_fails(monkeypatch, capturing):
    """An entry without workspace is called once more after torch's cache was emptied, but not while a graph is captured."""
    said = []

    def entry(*args):
        said.append("call")
        return fx.FXTX_ERR_ALLOC if said.count("call") == 1 else fx.FXTX_OK

    entry.__name__ = "entry"
    monkeypatch.setattr(layers, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "empty_cache", lambda: said.append("empty"))
    if capturing:
        with pytest.raises(fx.FxtxError):
            layers._call(entry, 0, 1, 2)
        assert said == ["call"]
    else:
        layers._call(entry, 0, 1, 2)
        assert said == ["call", "empty", "call"]


def test_a_call_that_stays_without_workspace_fails(monkeypatch):
    def entry(*args):
        return fx.FXTX_ERR_ALLOC

    monkeypatch.setattr(layers, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "empty_cache", lambda: None)
    with pytest.raises(fx.FxtxError) as e:
        layers._call(entry, 0)
    assert e.value.status == fx.FXTX_ERR_ALLOC
