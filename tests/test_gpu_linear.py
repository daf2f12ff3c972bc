"""The fused linear layer and its gradient against plain fp64 products, over types, layouts, sizes from one row up, odd
pitches and empty sums; the gradient against differences of the layer itself; the refusals of both.

Tolerances. A result is within c u S + w |result| of the exact one: u = 2^-24 (fp32 sums), S the sum of the magnitudes of
its terms, w the unit roundoff of the stored type. For a sum of K terms in fp32, however it is split, the error is at most
about K u S in the worst case and near sqrt(K) u S for rounding errors of either sign; c = 8 + 4 sqrt(K) is taken, with the
fp32 products' three-term split (2^-24 a term at most) inside the 8. An activation has a slope of at most 1.13, and fp32
evaluation adds a few u of its magnitude and of its input's: 32 u (1 + |z|). D is rounded to the type before the products
of the gradient: w of each term on top.
"""
import math

import pytest
import torch

import dense_linear_algebra_gb300 as fx

U = 2.0**-24
W_OF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0**-25}  # half the smallest float16
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def act64(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return torch.sigmoid(z) if act == "sigmoid" else z


def slope64(act, z):
    if act == "none":
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    (d,) = torch.autograd.grad(act64(act, z).sum(), z)
    return torch.where(z <= 0, torch.zeros_like(d), d).detach() if act == "relu" else d


def make(shape, dtype, seed, scale=1.0, pitch=None, offset=0):
    """A matrix of normal values; with a pitch, a column slice of a wider one (poisoned around it)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)
    if pitch is None:
        return x
    wide = torch.full((shape[0], pitch), float("nan"), dtype=dtype, device="cuda")
    wide[:, offset:offset + shape[1]] = x
    return wide[:, offset:offset + shape[1]]


def close(got, want, S, K, dtype, rounded=0.0):
    """`rounded`: the sum of the magnitudes of terms that were rounded to the type beforehand."""
    tol = (8 + 4 * math.sqrt(max(K, 1))) * U * S + W_OF[dtype] * (want.abs() + rounded) + TINY[dtype]
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off; first at {bad.nonzero()[0].tolist()}, worst "
                           f"{float((err / tol).nan_to_num(1e9).max()):.3g} of the tolerance")


def check_linear(m, n, k, dtype, act="none", bias=True, residual=True, w_t=False, pitch=0, offset=0, seed=0):
    p = lambda cols: None if not pitch else cols + pitch  # noqa: E731
    X = make((m, n), dtype, seed + 1, pitch=p(n), offset=offset)
    W = make((k, n) if w_t else (n, k), dtype, seed + 2, 1 / math.sqrt(max(n, 1)), pitch=p(n if w_t else k), offset=offset)
    W = W.t() if w_t else W
    b = make((1, k), dtype, seed + 3)[0] if bias else None
    R = make((m, k), dtype, seed + 4, pitch=p(k), offset=offset) if residual else None
    keep = make((m, k), dtype, seed + 5, pitch=p(k), offset=offset) if pitch else True
    out = make((m, k), dtype, seed + 6, pitch=p(k), offset=offset) if pitch else None
    out, pre = fx.linear(X, W, b, act=act, residual=R, pre=keep, out=out)
    again = fx.linear(X, W, b, act=act, residual=R)
    torch.cuda.synchronize()
    assert fx.device_error() == fx.FXTX_OK
    x, w = X.double(), W.double()
    z, S = x @ w, x.abs() @ w.abs()
    if bias:
        z, S = z + b.double(), S + b.double().abs()
    close(pre, z, S, n, dtype)
    want = act64(act, z)
    S = 1.13 * S + 4 * (1 + z.abs())
    if residual:
        want, S = want + R.double(), S + R.double().abs()
    close(out, want, S, n, dtype)
    assert torch.equal(out, again)  # the same bits on every call, kept Z or not
    if pitch and pitch > offset:  # what lies around the slices is untouched
        base = out._base if out._base is not None else out
        assert torch.isnan(base[:, :offset]).all() and torch.isnan(base[:, offset + k:]).all()


def check_grad(m, n, k, dtype, act="none", w_t=False, pitch=0, offset=0, seed=0):
    p = lambda cols: None if not pitch else cols + pitch  # noqa: E731
    X = make((m, n), dtype, seed + 1, pitch=p(n), offset=offset)
    W = make((k, n) if w_t else (n, k), dtype, seed + 2, 1 / math.sqrt(max(n, 1)), pitch=p(n if w_t else k), offset=offset)
    W = W.t() if w_t else W
    G = make((m, k), dtype, seed + 3, pitch=p(k), offset=offset)
    Z = make((m, k), dtype, seed + 4, pitch=p(k), offset=offset)
    dX, dW, db = fx.linear_grad(G, X, W, pre=Z, act=act)
    torch.cuda.synchronize()
    assert fx.device_error() == fx.FXTX_OK
    x, w = X.double(), W.double()
    d = G.double() * slope64(act, Z.double())
    # the slope's fp32 evaluation: 4 (1 + |z|) |G|, times 8 u at least
    S = d.abs() + (0.0 if act == "none" else 4 * G.double().abs() * (1 + Z.double().abs()))
    R = d.abs() * (act != "none")
    tiny = TINY[dtype] * (act != "none")  # D's rounding where it is a subnormal float16
    close(dX, d @ w.t(), (S + tiny / U) @ w.abs().t(), k, dtype, R @ w.abs().t())
    close(dW, x.t() @ d, x.abs().t() @ (S + tiny / U), m, dtype, x.abs().t() @ R)
    close(db, d.sum(0), S.sum(0), m, dtype)
    assert dW.stride() == ((1, n) if w_t else (k, 1)) or 1 in (n, k)


# around the kernels' borders: 64 features and outputs, 8 and 16 rows of float32, 128 rows, 256 x 256 tiles and more tiles
# than SMs
BORDERS = [(8, 300, 96), (9, 260, 200), (16, 100, 700), (17, 65, 300), (5, 2500, 70), (6, 70, 5000), (64, 64, 65), (64, 65, 64),
           (129, 300, 160), (700, 200, 2600), (2304, 520, 2560), (5000, 136, 1000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("shape", BORDERS, ids=str)
def test_kernel_borders(shape, w_t, dtype):
    check_linear(*shape, dtype, act=ACTS[sum(shape) % 6], w_t=w_t)
    check_grad(*shape, dtype, act=ACTS[(sum(shape) + 1) % 6], w_t=w_t)


SHAPES = [(1, 1, 1), (1, 64, 8), (2, 33, 17), (5, 128, 40), (16, 256, 136), (17, 1000, 24), (64, 96, 257), (65, 80, 64),
          (127, 129, 131), (128, 64, 256), (200, 520, 264), (300, 72, 1032), (1030, 48, 48), (4099, 32, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(shape, w_t, dtype):
    check_linear(*shape, dtype, act=ACTS[sum(shape) % 6], w_t=w_t)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(3, 200, 72), (130, 136, 192)], ids=str)
def test_linear_activations(shape, act, dtype):
    check_linear(*shape, dtype, act=act, bias=True, residual=False)
    check_linear(*shape, dtype, act=act, bias=False, residual=True, w_t=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pitch,offset", [(8, 0), (16, 8), (8, 4), (5, 3), (1, 1)])
@pytest.mark.parametrize("shape", [(1, 136, 80), (9, 264, 128), (150, 72, 200)], ids=str)
def test_linear_slices(shape, pitch, offset, dtype):
    """Column slices: aligned and unaligned starts and pitches, nothing written outside them."""
    check_linear(*shape, dtype, act="silu", pitch=pitch, offset=offset)
    check_linear(*shape, dtype, act="relu", pitch=pitch, offset=offset, w_t=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(1, 4096, 512), (4, 20_000, 64), (32, 5000, 1000), (700, 9000, 40), (2, 64, 20_000),
                                   (20_000, 40, 16), (513, 2049, 511)], ids=str)
def test_linear_long(shape, dtype):
    """Long sums, wide results and many rows."""
    check_linear(*shape, dtype, act="gelu", w_t=False)
    check_linear(*shape, dtype, act="none", w_t=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_linear_empty_and_in_place(dtype):
    b, R = make((1, 24), dtype, 1)[0], make((7, 24), dtype, 2)
    X, W = torch.empty(7, 0, dtype=dtype, device="cuda"), torch.empty(0, 24, dtype=dtype, device="cuda")
    out = fx.linear(X, W, b, act="relu", residual=R)
    assert torch.equal(out, (b.float().clamp(min=0) + R.float()).to(dtype))
    assert fx.linear(torch.empty(0, 5, dtype=dtype, device="cuda"), make((5, 24), dtype, 3)).shape == (0, 24)
    assert fx.linear(make((5, 5), dtype, 3), torch.empty(5, 0, dtype=dtype, device="cuda")).shape == (5, 0)
    for m in (3, 200):
        X, W, R = make((m, 96), dtype, 4), make((96, 72), dtype, 5), make((m, 72), dtype, 6)
        want = fx.linear(X, W, act="silu", residual=R)
        assert fx.linear(X, W, act="silu", residual=R, out=R) is R
        assert torch.equal(R, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("m", [2, 300])
def test_linear_non_finite_stays_in_its_row(m, dtype):
    """An infinity or a NaN in a row of X reaches that row of the result and no other."""
    X, W = make((m, 200), dtype, 1), make((200, 136), dtype, 2)
    want = fx.linear(X, W)
    X[1, 70] = float("inf")
    got = fx.linear(X, W)
    assert torch.isinf(got[1]).all()
    X[1, 70] = float("nan")
    got = fx.linear(X, W, act="relu")
    assert torch.isnan(got[1]).all()
    rest = [i for i in range(m) if i != 1]
    assert torch.equal(got[rest], want[rest].clamp(min=0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("w_t", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_grad_shapes(shape, w_t, dtype):
    check_grad(*shape, dtype, act=ACTS[(sum(shape) + 1) % 6], w_t=w_t)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ACTS)
def test_grad_activations(act, dtype):
    check_grad(130, 136, 192, dtype, act=act)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pitch,offset", [(8, 0), (16, 8), (8, 4), (5, 3)])
def test_grad_slices(pitch, offset, dtype):
    check_grad(150, 72, 200, dtype, act="silu", pitch=pitch, offset=offset)
    check_grad(40, 264, 88, dtype, act="none", pitch=pitch, offset=offset, w_t=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(30_000, 32, 32), (50_001, 24, 17), (300, 4000, 1000), (3, 20_000, 64)], ids=str)
def test_grad_long(shape, dtype):
    check_grad(*shape, dtype, act="gelu")
    check_grad(*shape, dtype, act="none", w_t=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_grad_empty_and_partial(dtype):
    X, W, G = (torch.empty(0, 5, dtype=dtype, device="cuda"), make((5, 6), dtype, 1),
               torch.empty(0, 6, dtype=dtype, device="cuda"))
    dX, dW, db = fx.linear_grad(G, X, W)
    assert dX.shape == (0, 5) and not dW.any() and not db.any()
    X, G = torch.empty(4, 0, dtype=dtype, device="cuda"), make((4, 6), dtype, 2)
    dX, dW, db = fx.linear_grad(G, X, torch.empty(0, 6, dtype=dtype, device="cuda"))
    assert dX.shape == (4, 0) and dW.shape == (0, 6)
    assert torch.allclose(db.float(), G.float().sum(0), atol=0.05)
    dX, dW, db = fx.linear_grad(torch.empty(4, 0, dtype=dtype, device="cuda"), make((4, 5), dtype, 3),
                                torch.empty(5, 0, dtype=dtype, device="cuda"))
    assert not dX.any() and dW.shape == (5, 0) and db.shape == (0,)
    G, X, W, Z = make((90, 48), dtype, 4), make((90, 40), dtype, 5), make((40, 48), dtype, 6), make((90, 48), dtype, 7)
    full = fx.linear_grad(G, X, W, pre=Z, act="gelu")
    for i in range(3):
        need = tuple(j == i for j in range(3))
        part = fx.linear_grad(G, X, W, pre=Z, act="gelu", need=need)
        assert torch.equal(part[i], full[i]) and [p is None for p in part] == [not x for x in need]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_grad_against_differences(act):
    """fp32: the gradient of sum(G * linear(X, W, b)) against central differences of the layer, in directions of X, W and
    b. A step h leaves h^2/6 of a third derivative (at most 2 in size over the activations, times the cube of the
    direction's change in z) and 2 u S / h of the two fp32 layers; relu's kinks within the step are left out."""
    m, n, k, h = 24, 20, 28, 2.0**-6
    X, W, b, G = make((m, n), torch.float32, 1), make((n, k), torch.float32, 2, 0.3), make((1, k), torch.float32, 3)[0], \
        make((m, k), torch.float32, 4)
    out, Z = fx.linear(X, W, b, act=act, pre=True)
    for which, d in (("X", make((m, n), torch.float32, 5)), ("W", make((n, k), torch.float32, 6)),
                     ("b", make((1, k), torch.float32, 7)[0])):
        up = fx.linear(X + h * d if which == "X" else X, W + h * d if which == "W" else W,
                       b + h * d if which == "b" else b, act=act)
        down = fx.linear(X - h * d if which == "X" else X, W - h * d if which == "W" else W,
                         b - h * d if which == "b" else b, act=act)
        if which == "b":
            dz = d.double().expand(m, k)
        else:
            dz = d.double() @ W.double() if which == "X" else X.double() @ d.double()
        g = G.clone()
        if act == "relu":
            g[(Z.double().abs() <= 1.01 * h * dz.abs() + 1e-5)] = 0
        diff = (g.double() * (up.double() - down.double())).sum() / (2 * h)
        dX, dW, db = fx.linear_grad(g, X, W, pre=Z, act=act)
        got = ({"X": dX, "W": dW, "b": db}[which].double() * d.double()).sum()
        S = (g.double().abs() * (X.double().abs() @ W.double().abs() + b.double().abs() + 1)).sum()
        tol = h * h / 3 * (g.double().abs() * dz.abs() ** 3).sum() + 64 * U * S / h
        assert abs(float(diff - got)) <= float(tol)


@pytest.mark.gpu
def test_other_stream():
    X, W = make((200, 96), torch.bfloat16, 1), make((96, 72), torch.bfloat16, 2)
    want, wZ = fx.linear(X, W, act="gelu", pre=True)
    grads = fx.linear_grad(want, X, W, pre=wZ, act="gelu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, Z = fx.linear(X, W, act="gelu", pre=True, stream=side)
    got = fx.linear_grad(out, X, W, pre=Z, act="gelu", stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((out, Z, *got), (want, wZ, *grads)):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_graph_capture(dtype):
    """A layer and its gradient in a CUDA graph, replayed on new inputs."""
    X, W, b = make((96, 128), dtype, 1), make((128, 200), dtype, 2, 0.1), make((1, 200), dtype, 3)[0]

    def step():
        out, Z = fx.linear(X, W, b, act="silu", pre=True)
        return (out, Z) + fx.linear_grad(out, X, W, pre=Z, act="silu")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    X.copy_(make((96, 128), dtype, 9))
    graph.replay()
    got = [t.clone() for t in held]
    for x, y in zip(got, step()):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_no_workspace_is_reported(monkeypatch):
    """float32 operands need a workspace: without one the call fails with its status, and the next one works."""
    X, W = make((100, 300), torch.float32, 1), make((300, 200), torch.float32, 2)
    want = fx.linear(X, W)
    monkeypatch.setenv("FXTX_FAIL_ALLOC", "1")
    with pytest.raises(fx.FxtxError) as e:
        fx.linear(X, W)
    assert e.value.status == fx.FXTX_ERR_ALLOC
    monkeypatch.delenv("FXTX_FAIL_ALLOC")
    assert torch.equal(fx.linear(X, W), want)


@pytest.mark.gpu
def test_python_refusals():
    X, W, b = make((6, 8), torch.float32, 1), make((8, 4), torch.float32, 2), make((1, 4), torch.float32, 3)[0]
    G = make((6, 4), torch.float32, 4)
    for call in (lambda: fx.linear(X[0], W), lambda: fx.linear(X, W[:7]), lambda: fx.linear(X, W.half()),
                 lambda: fx.linear(X, W, b[:3]), lambda: fx.linear(X, W, b, act="softmax"),
                 lambda: fx.linear(X, W, residual=G[:5]), lambda: fx.linear(X, W, out=G[:, :3]),
                 lambda: fx.linear(X, W, pre=G.t()), lambda: fx.linear(X.t().contiguous().t(), W),
                 lambda: fx.linear(X[:1].expand(6, 8), W), lambda: fx.linear(X, make((8, 8), torch.float32, 5)[:, ::2]),
                 lambda: fx.linear(X.cpu(), W), lambda: fx.linear(X, W.cpu()),
                 lambda: fx.linear_grad(G, X, W, act="gelu"), lambda: fx.linear_grad(G[:5], X, W),
                 lambda: fx.linear_grad(G, X, W, pre=G[:5], act="gelu"), lambda: fx.linear_grad(G.half(), X, W)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fx.linear(X.double(), W.double())


def test_host_tensors_are_refused():
    X, W = torch.zeros(3, 4), torch.zeros(4, 5)
    with pytest.raises(ValueError):
        fx.linear(X, W)
    with pytest.raises(ValueError):
        fx.linear_grad(torch.zeros(3, 5), X, W)


def test_c_refusals():
    """Refused before any device work; the pointers are never read."""
    bad, ok = fx.FXTX_ERR_INVALID_ARG, fx.FXTX_OK

    def lin(type=1, m=4, n=8, k=6, X=16, ldx=8, W=16, ldw=6, tr=0, b=None, act=0, R=None, ldr=0, Z=None, ldz=0, OUT=16,
            ldo=6):
        return fx.fxtx_linear(type, m, n, k, X, ldx, W, ldw, tr, b, act, R, ldr, Z, ldz, OUT, ldo, None)

    for kw in (dict(type=3), dict(act=6), dict(act=-1), dict(m=-1), dict(n=-1), dict(k=1 << 31), dict(ldx=7), dict(ldw=5),
               dict(tr=2), dict(tr=1, ldw=7), dict(X=None), dict(W=None), dict(OUT=None), dict(ldo=5), dict(R=16, ldr=5),
               dict(Z=16, ldz=5)):
        assert lin(**kw) == bad, kw
    assert lin(m=0, X=None, OUT=None) == ok and lin(k=0, W=None, OUT=None) == ok

    def grad(type=1, m=4, n=8, k=6, G=16, ldg=6, X=16, ldx=8, W=16, ldw=6, tr=0, Z=16, ldz=6, act=2, DX=16, lddx=8, DW=16,
             lddw=6, DB=16):
        return fx.fxtx_linear_grad(type, m, n, k, G, ldg, X, ldx, W, ldw, tr, Z, ldz, act, DX, lddx, DW, lddw, DB, None)

    for kw in (dict(type=-1), dict(act=7), dict(m=-1), dict(ldg=5), dict(G=None), dict(Z=None), dict(ldz=5), dict(lddx=7),
               dict(lddw=5), dict(X=None), dict(W=None), dict(ldx=7), dict(tr=1, ldw=8, lddw=7), dict(tr=3)):
        assert grad(**kw) == bad, kw
    assert grad(DX=None, DW=None, DB=None) == ok and grad(n=0, DB=None, ldx=0, lddx=0) == ok


def test_no_device_is_reported_as_unsupported():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert fx.fxtx_linear(1, 4, 8, 6, 16, 8, 16, 6, 0, None, 0, None, 0, None, 0, 16, 6, None) == fx.FXTX_ERR_UNSUPPORTED
