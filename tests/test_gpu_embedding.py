"""The embedding lookup bit for bit against fp32 indexing, and its gradient against sums in 64 bits: every size at which the
sort or the sums take another way, ids of all distributions, ids outside the table, odd pitches.

Tolerance of a row of c terms: fp32 sums, (8 + 4 sqrt(c)) 2^-24 of the sum of the terms' magnitudes, and the unit roundoff
of the stored type.
"""
import math

import pytest
import torch

import dense_linear_algebra_gb300 as fx

pytestmark = pytest.mark.gpu

U = 2.0**-24
W_OF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0**-25}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def normal(shape, dtype, seed, pad=0, offset=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    if not pad:
        return x
    wide = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, offset:offset + shape[1]] = x
    return wide[:, offset:offset + shape[1]]


def ids_of(kind, m, count, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if kind == "uniform":
        return torch.randint(0, count, (m,), generator=gen, device="cuda")
    if kind == "one":
        return torch.full((m,), count // 2, device="cuda")
    if kind == "sorted":
        return torch.arange(m, device="cuda") * count // max(m, 1)
    if kind == "falling":
        return torch.arange(m, device="cuda").flip(0) % count
    u = torch.rand(m, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(count + 1)).long().sub_(1).clamp_(0, count - 1)
    if kind == "padded":
        drop = torch.rand(m, generator=gen, device="cuda") < 0.3
        ids = torch.where(drop, torch.where(u < 0.5, -1, count), ids)
    return ids


def check_lookup(ids, count, n, dtype, scale=1.0, pad=0, offset=0):
    E = normal((count, n), dtype, 1, pad, offset)
    out = normal((ids.shape[0], n), dtype, 2, pad, offset) if pad else None
    got = fx.embedding(ids, E, scale=scale, out=out)
    inside = (ids >= 0) & (ids < count)
    rows = E[torch.where(inside, ids, 0)] if count else torch.zeros((ids.shape[0], n), dtype=dtype, device="cuda")
    want = torch.where(inside[:, None], (rows.float() * torch.tensor(scale, device="cuda")).to(dtype), torch.zeros_like(rows))
    assert torch.equal(got, want)
    if pad:
        assert torch.isnan(got._base[:, :offset]).all() and torch.isnan(got._base[:, offset + n:]).all()


def check_gradient(ids, count, n, dtype, scale=1.0, pad=0, offset=0):
    m = ids.shape[0]
    G = normal((m, n), dtype, 1, pad, offset)
    inside = (ids >= 0) & (ids < count)
    G[~inside] = float("nan")  # a row that has no id is not taken
    out = normal((count, n), dtype, 2, pad, offset) if pad else None
    got = fx.embedding_grad(G, ids, count, scale=scale, out=out)
    again = fx.embedding_grad(G, ids.int(), count, scale=scale)
    torch.cuda.synchronize()
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    g = G[inside].double() * s32
    at = ids[inside].long()
    want = torch.zeros((count, n), dtype=torch.float64, device="cuda").index_add_(0, at, g)
    S = torch.zeros_like(want).index_add_(0, at, g.abs())
    c = torch.zeros(count, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    tol = (8 + 4 * c.sqrt())[:, None] * U * S + W_OF[dtype] * 1.001 * want.abs() + TINY[dtype]
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"
    assert torch.equal(got, again)
    if pad:
        assert torch.isnan(got._base[:, :offset]).all() and torch.isnan(got._base[:, offset + n:]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 3, 8, 32, 100, 256, 301, 1024, 2056, 4096, 8200, 20_001])
def test_widths(n, dtype):
    ids = ids_of("padded", 133, 57, n)
    check_lookup(ids, 57, n, dtype, scale=math.sqrt(n))
    check_gradient(ids, 57, n, dtype, scale=math.sqrt(n))


@pytest.mark.parametrize("kind", ["uniform", "one", "sorted", "falling", "frequent", "padded"])
@pytest.mark.parametrize("m", [0, 1, 2, 31, 32, 33, 64, 65, 255, 257, 2047, 2048, 2049, 1023, 1024, 1025, 4097, 8192, 8193, 16_383, 16_384, 16_385, 65_537])
def test_numbers_of_ids(m, kind):
    for count in (1, 300, 5000):
        ids = ids_of(kind, m, count, m + count)
        check_lookup(ids, count, 24, torch.float32)
        check_gradient(ids, count, 24, torch.float32)


@pytest.mark.parametrize("count", [1, 2, 3, 255, 256, 511, 512, 513, 1023, 1024, 65_535, 65_536, 262_143, 262_144, 300_000, 20_000_000])
@pytest.mark.parametrize("m", [5, 3000, 12_000, 66_000])
def test_sizes_of_the_table(count, m):
    """Every number of bits an id may have, in both sorts: one to three passes."""
    ids = ids_of("uniform", m, count, 7)
    ids[:4] = torch.tensor([0, count - 1, count, -1], device="cuda")
    check_lookup(ids, count, 4, torch.float32)
    check_gradient(ids, count, 4, torch.float32, scale=0.5)


def test_no_table():
    ids = torch.tensor([0, 1, -1], device="cuda")
    assert torch.equal(fx.embedding(ids, torch.empty((0, 16), device="cuda")), torch.zeros((3, 16), device="cuda"))
    assert fx.embedding_grad(torch.ones((3, 16), device="cuda"), ids, 0).shape == (0, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (1, 0), (5, 3)])
@pytest.mark.parametrize("n", [32, 301])
def test_column_slices(n, pad, offset, dtype):
    ids = ids_of("padded", 300, 90, 5)
    check_lookup(ids, 90, n, dtype, pad=pad, offset=offset)
    check_gradient(ids, 90, n, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_frequent_id_of_many_rows(dtype):
    """200,000 rows of one id among others: three levels of partial sums."""
    ids = ids_of("frequent", 262_144, 1000, 3)
    ids[30_000:230_000] = 17
    check_gradient(ids, 1000, 40, dtype, scale=2.0)


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
def test_ids_far_outside(bits):
    ids = torch.tensor([3, 2**31 - 1, -2**31, 1, 4, 5], dtype=bits, device="cuda")
    if bits is torch.int64:
        ids[4], ids[5] = 2**32 + 1, -2**63  # 1 in its lower half
    E = normal((4, 40), torch.float32, 1)
    got = fx.embedding(ids, E)
    assert torch.equal(got[0], E[3]) and torch.equal(got[3], E[1])
    assert not got[1].any() and not got[2].any() and not got[4].any() and not got[5].any()
    G = normal((6, 40), torch.float32, 2)
    dE = fx.embedding_grad(G, ids, 4)
    assert torch.equal(dE[3], G[0]) and torch.equal(dE[1], G[3]) and not dE[0].any() and not dE[2].any()


def test_values_that_are_not_finite_stay_in_their_row():
    ids = torch.tensor([2, 0, 2, 1] * 50, device="cuda")
    G = normal((200, 64), torch.float32, 1)
    want = fx.embedding_grad(G, ids, 4)
    G[0, 7] = float("inf")
    got = fx.embedding_grad(G, ids, 4)
    assert torch.isinf(got[2, 7])
    want[2, 7] = got[2, 7]
    assert torch.equal(got, want)


def test_streams_and_graphs():
    for m in (900, 10_000, 30_000):
        ids, other = ids_of("frequent", m, 700, 1), ids_of("padded", m, 700, 2)
        E, G = normal((700, 72), torch.bfloat16, 1), normal((m, 72), torch.bfloat16, 2)
        side = torch.cuda.Stream()
        want = fx.embedding(ids, E), fx.embedding_grad(G, ids, 700)
        side.wait_stream(torch.cuda.current_stream())
        got = fx.embedding(ids, E, stream=side), fx.embedding_grad(G, ids, 700, stream=side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = fx.embedding(ids, E), fx.embedding_grad(G, ids, 700)
        want = fx.embedding(other, E), fx.embedding_grad(G, other, 700)
        ids.copy_(other)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
