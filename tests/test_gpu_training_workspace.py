"""Workspace of layer norm, the embedding lookup and cross entropy: calls without it fail and leave the next one whole; calls at once on
two streams, and graphs replayed at once, do not share theirs."""
import pytest
import torch

import dense_linear_algebra_gb300 as fx

pytestmark = pytest.mark.gpu


def inputs(m, n, k, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    return {"X": normal(m, n), "G": normal(m, n), "W": normal(k, n).t(), "b": normal(k),
            "ids": torch.randint(-1, k + 1, (m,), generator=gen, device="cuda")}


def calls(s):
    """Every operator once, on what `inputs` gives; all results."""
    k = s["b"].shape[0]
    u, mean, rstd = fx.layer_norm(s["X"], stats=True)
    out = [u, mean, rstd, *fx.layer_norm_grad(s["G"], s["X"], None, mean, rstd)]
    out += [fx.embedding(s["ids"], s["W"].t()), fx.embedding_grad(s["G"], s["ids"], k)]
    loss, lse = fx.cross_entropy(s["X"], s["W"], s["ids"], s["b"])
    return out + [loss, lse, *fx.cross_entropy_grad(s["X"], s["W"], s["ids"], lse, s["b"], g=0.5)]


SIZES = [(300, 200, 700, torch.bfloat16), (9, 96, 130, torch.float32), (3000, 32, 10, torch.float32), (2000, 40, 50, torch.float16),
         (20_000, 72, 300, torch.float16), (40, 2056, 1000, torch.float32)]


@pytest.mark.parametrize("m,n,k,dtype", SIZES)
def test_calls_without_workspace(m, n, k, dtype, monkeypatch):
    s = inputs(m, n, k, dtype, 1)
    want = calls(s)
    mean, rstd, lse = want[1], want[2], want[-4]
    monkeypatch.setenv("FXTX_FAIL_ALLOC", "1")
    for call in (lambda: fx.layer_norm_grad(s["G"], s["X"], None, mean, rstd), lambda: fx.embedding_grad(s["G"], s["ids"], k),
                 lambda: fx.cross_entropy(s["X"], s["W"], s["ids"], s["b"]),
                 lambda: fx.cross_entropy_grad(s["X"], s["W"], s["ids"], lse, s["b"])):
        try:
            call()  # (some sizes take none)
        except fx.FxtxError as e:
            assert e.status == fx.FXTX_ERR_ALLOC
    with pytest.raises(fx.FxtxError):
        fx.embedding_grad(s["G"], s["ids"], k)
    monkeypatch.delenv("FXTX_FAIL_ALLOC")
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, calls(s)))


@pytest.mark.parametrize("m,n,k,dtype", SIZES)
def test_calls_at_once(m, n, k, dtype):
    sets = [inputs(m, n, k, dtype, seed) for seed in (1, 2)]
    want = [calls(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(calls(s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("m,n,k,dtype", SIZES)
def test_graphs_at_once(m, n, k, dtype):
    sets = [inputs(m, n, k, dtype, seed) for seed in (1, 2)]
    want = [calls(s) for s in sets]
    graphs, got = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(calls(s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_behind_the_last_are_left_alone():
    """Outputs into the first rows of larger tensors."""
    m, n, k = 70, 96, 130
    s = inputs(m, n, k, torch.bfloat16, 1)
    wide = torch.full((m + 9, n), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fx.layer_norm(s["X"], out=wide[:m]), fx.layer_norm(s["X"])) and (wide[m:] == 7).all()
    wide.fill_(7)
    assert torch.equal(fx.embedding(s["ids"], s["W"].t(), out=wide[:m]), fx.embedding(s["ids"], s["W"].t())) and (wide[m:] == 7).all()
    table = torch.full((k + 9, n), 7.0, dtype=torch.bfloat16, device="cuda")
    fx.embedding_grad(s["G"], s["ids"], k, out=table[:k])
    assert torch.equal(table[:k], fx.embedding_grad(s["G"], s["ids"], k)) and (table[k:] == 7).all()
