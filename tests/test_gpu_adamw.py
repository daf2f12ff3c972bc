"""The AdamW step: 32-bit states against the formula in 64 bits, 8-bit states bit by bit against the formula in fp32
with every operation rounded on its own (numpy), and its refusals."""
import ctypes

import numpy as np
import pytest
import torch

import dense_linear_algebra_gb300 as fx

B = 256
U = 2.0**-24  # fp32 rounding
HALF = {torch.float32: U, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # unit roundoffs: 24, 8, 11 bits
H = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.02)


def _ref32(p, g, m, v, t, dtype, lr, betas, eps, weight_decay):
    """The step in `dtype` (numpy), every operation rounded on its own; constants rounded from double."""
    f = lambda x: np.asarray(x, dtype=dtype)  # noqa: E731
    b1, b2 = betas
    p, g, m, v = f(p), f(g), f(m), f(v)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    r = np.sqrt(v)
    step = m / (r * f(1 / np.sqrt(1 - b2**t)) + f(eps))
    p = p * f(1 - lr * weight_decay) - step * f(lr / (1 - b1**t))
    return p, m, v, r


def _blocks(x):
    n = x.size
    return np.pad(x, (0, -n % B)).reshape(-1, B)


def _encode(x, levels):
    """Codes and scales of each block of x, in fp32."""
    f = np.float32
    x = _blocks(x)
    top = np.abs(x).max(1)
    with np.errstate(all="ignore"):
        held = ~(top < f(1e-30))
        inv = np.where(held, f(1) / top * f(levels**2), f(0)).astype(f)
        scale = np.where(held, top * (f(1) / f(levels**2)), f(0)).astype(f)
        c = np.minimum(np.rint(np.sqrt(np.abs(x) * inv[:, None])), levels)
    c = np.nan_to_num(c, nan=0.0)
    c = np.where(x < 0, -c, c)
    if levels == 255:
        c = np.maximum(c, (x > 0).astype(f))
    return c, scale


def _decode(c, scale):
    with np.errstate(all="ignore"):
        return (c * np.abs(c)).astype(np.float32) * scale[:, None]


def _tensors(sizes, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale).to(dtype).cuda() for n in sizes]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


SIZES = [[1], [255, 256, 257], [7, 4096, 1, 70_001, 0, 33], [100_000] * 3, [3] * 500]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("p_type,g_type,c_type", [
    (torch.float32, torch.float32, None), (torch.float32, torch.bfloat16, torch.bfloat16),
    (torch.bfloat16, torch.bfloat16, None), (torch.float16, torch.float32, torch.float32),
    (torch.float32, torch.float16, torch.float16)])
def test_32_bit_states(sizes, p_type, g_type, c_type):
    """Three steps from zero states. m and v: four and five roundings of sums of like or unlike terms, so 8 U of the
    sum of the terms' magnitudes a step; p: as many again of the step's size, and one rounding to its type a step."""
    params = _tensors(sizes, p_type, 1)
    copies = None if c_type is None else [torch.zeros_like(p, dtype=c_type) for p in params]
    opt = fx.AdamW(params, copies=copies, **H)
    ref = [[_np(p), np.zeros(n), np.zeros(n)] for p, n in zip(params, sizes)]
    mag = [np.zeros(n) for n in sizes]
    for t in (1, 2, 3):
        grads = _tensors(sizes, g_type, 10 + t, 0.1 * t)
        opt.step(grads)
        torch.cuda.synchronize()
        for i, n in enumerate(sizes):
            g = _np(grads[i])
            p, m, v, r = _ref32(ref[i][0], g, ref[i][1], ref[i][2], t, np.float64, **H)
            mag[i] = 0.9 * mag[i] + 0.1 * np.abs(g)
            at = opt.offsets[i]
            got_m, got_v = _np(opt.exp_avg[at:at + n]), _np(opt.exp_avg_sq[at:at + n])
            assert np.all(np.abs(got_m - m) <= 8 * t * U * mag[i])
            assert np.all(np.abs(got_v - v) <= 8 * t * U * v)
            step = H["lr"] / (1 - 0.9**t) * mag[i] / (r / np.sqrt(1 - 0.999**t) + H["eps"])
            tol = 2 * U * np.abs(p) + 32 * t * U * step
            small = 2.0**-25 if p_type == torch.float16 else 0.0  # half the smallest step of float16
            assert np.all(np.abs(_np(params[i]) - p) <= tol + HALF[p_type] * np.abs(p) * 1.01 + small)
            if copies is not None:
                small = 2.0**-25 if c_type == torch.float16 else 0.0
                assert np.all(np.abs(_np(copies[i]) - p) <= tol + HALF[c_type] * np.abs(p) * 1.01 + small)
            # the next step starts from what is held
            ref[i] = [_np(params[i]), got_m, got_v]
    assert opt.steps == 3


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("p_type,g_type", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                           (torch.float16, torch.float32)])
def test_8_bit_states_bit_by_bit(sizes, p_type, g_type):
    """Codes, scales, moments and params are the fp32 formulas' to the last bit, over steps that decode what the last
    one held; zero blocks, and values far below their block's largest, among them."""
    params = _tensors(sizes, p_type, 2)
    opt = fx.AdamW(params, state_bits=8, **H)
    held = [(np.zeros((-(-n // B), B), np.float32), np.zeros(-(-n // B), np.float32)) * 2 for n in sizes]
    ref_p = [p.float().cpu().numpy() for p in params]
    for t in (1, 2, 3):
        grads = _tensors(sizes, torch.float32, 20 + t)
        for j, g in enumerate(grads):
            g.mul_(torch.logspace(-9, 1, g.numel(), device="cuda") if j % 2 else 1e-3)
            if g.numel() > 600:
                g[256:512] = 0
        grads = [g.to(g_type) for g in grads]
        opt.step(grads)
        got_m, got_v = opt.moments()
        torch.cuda.synchronize()
        for i, n in enumerate(sizes):
            mc, ms, rc, rs = held[i]
            m, r = _decode(mc, ms).reshape(-1)[:n], _decode(rc, rs).reshape(-1)[:n]
            p, m, v, r = _ref32(ref_p[i], grads[i].float().cpu().numpy(), m, r * r, t, np.float32, **H)
            held[i] = mc, ms, rc, rs = _encode(m, 127) + _encode(r, 255)
            p = torch.from_numpy(p).to(p_type)
            assert torch.equal(params[i].cpu(), p)
            ref_p[i] = p.float().numpy()
            at, nb = opt.offsets[i], -(-n // B)
            assert np.array_equal(opt.exp_avg[at:at + n].cpu().numpy(), mc.reshape(-1)[:n])
            assert np.array_equal(opt.exp_avg_sq[at:at + n].cpu().numpy(), rc.reshape(-1)[:n])
            assert np.array_equal(opt.exp_avg_scale[at // B:at // B + nb].cpu().numpy(), ms)
            assert np.array_equal(opt.exp_avg_sq_scale[at // B:at // B + nb].cpu().numpy(), rs)
            assert np.array_equal(got_m[at:at + n].cpu().numpy(), _decode(mc, ms).reshape(-1)[:n])
            x = _decode(rc, rs).reshape(-1)[:n]
            assert np.array_equal(got_v[at:at + n].cpu().numpy(), x * x)


@pytest.mark.gpu
def test_8_bit_codes_against_64_bits():
    """What is held is within half a code of the moments in 64 bits, in the root of a value over its scale; a root
    above zero is never held as zero. Half a code, and 127 (255) times a few fp32 roundings."""
    n = 10_000
    (p,), (g,) = _tensors([n], torch.float32, 5), _tensors([n], torch.float32, 6)
    g.mul_(torch.logspace(-8, 0, n, device="cuda"))
    opt = fx.AdamW([p], state_bits=8, **H)
    opt.step([g])
    g = _np(g)
    for x, codes, levels in ((0.1 * g, opt.exp_avg, 127), (np.sqrt(0.001) * np.abs(g), opt.exp_avg_sq, 255)):
        x, c = _blocks(x), _blocks(codes.cpu().numpy()[:n].astype(np.float64))
        want = np.sign(x) * np.sqrt(np.abs(x) / np.abs(x).max(1, keepdims=True)) * levels
        floor = (levels == 255) & (np.abs(want) < 0.5)
        assert np.all((np.abs(want - c) <= 0.5 + 1e-4) | (floor & (c == (x != 0))))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_unaligned_views_none_gradients_and_streams(bits):
    """Views at odd offsets, a missing gradient, and another stream give what aligned tensors give."""
    sizes = [1000, 513, 256, 77]
    base, gbase = torch.randn(4000, device="cuda"), torch.randn(4000, device="cuda")
    at = [1, 1006, 1523, 1801]
    odd, godd = [base[a:a + n] for a, n in zip(at, sizes)], [gbase[a:a + n] for a, n in zip(at, sizes)]
    even, geven = [t.clone() for t in odd], [t.clone() for t in godd]
    godd[2] = geven[2] = None
    keep = base.clone()
    a, b = fx.AdamW(odd, state_bits=bits, **H), fx.AdamW(even, state_bits=bits, **H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(godd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.step(geven)
    for x, y in zip(odd, even):
        assert torch.equal(x, y)
    for x, y in zip(a.moments(), b.moments()):
        assert torch.equal(x, y)
    assert torch.equal(odd[2], keep[1523:1523 + 256])
    touched = torch.zeros(4000, dtype=torch.bool, device="cuda")
    for i, n in enumerate(sizes):
        touched[at[i]:at[i] + n] = i != 2
    assert torch.equal(base[~touched], keep[~touched])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_non_finite_gradients_stay_in_their_block(bits):
    """An infinity or a NaN makes NaN of its element (32 bits) or of its block's moments (8 bits), and of nothing else."""
    (p,) = _tensors([2000], torch.float32, 7)
    (g,) = _tensors([2000], torch.float32, 8)
    clean_p, clean_g = p.clone(), g.clone()
    g[300], g[700] = float("inf"), float("nan")
    a, b = fx.AdamW([p], state_bits=bits, **H), fx.AdamW([clean_p], state_bits=bits, **H)
    for _ in range(2):
        a.step([g])
        b.step([clean_g])
    bad = torch.zeros(2000, dtype=torch.bool, device="cuda")
    if bits == 32:
        bad[300] = bad[700] = True
    else:
        bad[256:768] = True
    assert torch.equal(p[~bad], clean_p[~bad])
    assert torch.equal(a.moments()[0][:2000][~bad], b.moments()[0][:2000][~bad])
    assert torch.isnan(p[[300, 700]]).all()
    if bits == 8:
        assert torch.isnan(a.moments()[0][256:768]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_state_dict_resumes(bits):
    sizes = [700, 300]
    p1 = _tensors(sizes, torch.float32, 3)
    p2 = [t.clone() for t in p1]
    a, b = fx.AdamW(p1, state_bits=bits, **H), fx.AdamW(p2, state_bits=bits, **H)
    for t in range(4):
        grads = _tensors(sizes, torch.float32, 30 + t)
        a.step(grads)
        b.step(grads)
        if t == 1:  # b goes on from what it saved
            saved = b.state_dict()
            b = fx.AdamW(p2, state_bits=bits, **H)
            b.load_state_dict(saved)
    assert b.steps == 4
    for x, y in zip(p1, p2):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_python_refusals():
    p = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        fx.AdamW([])
    with pytest.raises(ValueError):
        fx.AdamW([p], state_bits=16)
    with pytest.raises(TypeError):
        fx.AdamW([p.double()])
    with pytest.raises(ValueError):
        fx.AdamW([p.view(8, 8).t()])
    with pytest.raises(ValueError):
        fx.AdamW([p, p.half()])
    with pytest.raises(ValueError):
        fx.AdamW([p], copies=[p[:63]])
    opt = fx.AdamW([p])
    for grads in ([], [None], [p[:63]], [p, p], [p.cpu()], [p.view(8, 8).t()]):
        with pytest.raises(ValueError):
            opt.step(grads)
    with pytest.raises(TypeError):
        opt.step([p.double()])
    opt.lr = -1.0
    with pytest.raises(fx.FxtxError):
        opt.step([p])
    with pytest.raises(ValueError):
        opt.load_state_dict(fx.AdamW([p[:1], p[1:60].clone()], state_bits=8).state_dict())
    assert opt.steps == 0 and not p.any()


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        fx.AdamW([torch.zeros(4)])


def test_c_refusals():
    """Refused before any device work."""
    row = np.zeros((1, 8), np.int64)
    row[0] = [8, 16, 16, 16, 16, 16, 16, 0]

    def call(count=1, table=row, p=0, g=0, c=0, bits=32, step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0):
        return fx.fxtx_adamw(count, None if table is None else table.ctypes.data, p, g, c, bits, step, lr, b1, b2, eps,
                             wd, None)

    bad = fx.FXTX_ERR_INVALID_ARG
    nan = float("nan")
    for kw in (dict(count=-1), dict(table=None), dict(p=3), dict(g=-1), dict(c=9), dict(bits=4), dict(step=0),
               dict(lr=-1.0), dict(lr=nan), dict(b1=1.0), dict(b2=nan), dict(b2=-0.1), dict(eps=-1.0),
               dict(wd=float("inf"))):
        assert call(**kw) == bad, kw
    for col in (1, 2, 3, 4):
        t = row.copy()
        t[0, col] = 0
        assert call(table=t) == bad
    t = row.copy()
    t[0, 5] = 0
    assert call(table=t, bits=8) == bad
    t = row.copy()
    t[0, 0] = -1
    assert call(table=t) == bad
    t[0, 0] = (1 << 39) + 1
    assert call(table=t) == bad
    t[0] = 0
    assert call(table=t) == fx.FXTX_OK and call(count=0, table=None) == fx.FXTX_OK
    assert fx.fxtx_adamw_moments(-1, *([None] * 7)) == bad
    assert fx.fxtx_adamw_moments(8, *([None] * 7)) == bad
    assert fx.fxtx_adamw_moments(0, *([None] * 7)) == fx.FXTX_OK
    assert ctypes.sizeof(ctypes.c_int64) * 8 == row.strides[0]
