"""The activations and their slopes alone, against 64 bits: a layer of one feature and one output with W = 1 shows the
activation of X itself (the sum of one term is exact in every type), and its gradient with G = 1, where n = k = 1, the slope.

Tolerances, in units u = 2^-24 of the quantity named: an exponential of float32 layers is within 2 u, a reciprocal 2 u, each
product, sum and constant 1 u, the polynomial of erfc 6 u; 16 u of the value cover the longest chain but gelu's, which has 24.
gelu_tanh's argument v is rounded three times and its exponential carries that over: 4 |v| u more. A slope that is a difference of two
terms is held to that many units of the terms' sum. 16-bit layers round the result once more (w) and take the short
exponential, whose argument is rounded twice and whose own error is 1.2 |x| + 2 units: 4 |x| u more. Values below 2^-120 may
be zero, and float16 ends at 2^-25.
"""
import math

import pytest
import torch

import dense_linear_algebra_gb300 as fx

pytestmark = pytest.mark.gpu

U = 2.0**-24
W_OF = {torch.float32: 0.0, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 2.0**-120, torch.bfloat16: 2.0**-120, torch.float16: 2.0**-25}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
C0, C1 = math.sqrt(2 / math.pi), 0.044715


def values(act, z):
    """In 64 bits: the activation, the sum of its slope's terms in magnitude, the slope, the exponential's argument."""
    phi = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z.abs() * phi, cdf + z * phi, 0.5 * z * z
    v, dv = z, torch.ones_like(z)
    if act == "gelu_tanh":
        v, dv = 2 * C0 * (z + C1 * z**3), 2 * C0 * (1 + 3 * C1 * z * z)
    e = torch.exp(-v.abs())
    s, rest = torch.where(v < 0, e, torch.ones_like(e)) / (1 + e), torch.where(v < 0, torch.ones_like(e), e) / (1 + e)
    if act == "sigmoid":
        return s, s * rest, s * rest, v
    return z * s, s + (z * s * rest * dv).abs(), s + z * s * rest * dv, v


def tolerance(act, dtype, size, x):
    units = (24 if act == "gelu" else 16) + (4 * x.abs() if act == "gelu_tanh" or dtype != torch.float32 else 0)
    return (units * U + W_OF[dtype]) * size + TINY[dtype]


def points(dtype, span):
    z = torch.cat([torch.linspace(-span, span, 40_001), torch.logspace(-30, 0, 301), -torch.logspace(-30, 0, 301)])
    return z.to(dtype).cuda()


def check(got, want, tol, z):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first at z = {float(z[bad][0])}: {float(got[bad][0])}, not {float(want[bad][0])}"


def act_of(z, act):
    return fx.linear(z[:, None], torch.ones(1, 1, dtype=z.dtype, device="cuda"), act=act)[:, 0]


def slope_of(z, act):
    one = torch.ones_like(z)[:, None]
    return fx.linear_grad(one, one, one[:1], pre=z[:, None], act=act, need=(True, False, False))[0][:, 0]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("span", [1.0, 6.0, 13.0])
def test_gelu(dtype, span):
    z = points(dtype, span)
    a, size, s, x = values("gelu", z.double())
    check(act_of(z, "gelu"), a, tolerance("gelu", dtype, a.abs(), x), z)
    check(slope_of(z, "gelu"), s, tolerance("gelu", dtype, size, x), z)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act,span", [("sigmoid", 80.0), ("sigmoid", 20.0), ("silu", 80.0), ("silu", 10.0),
                                      ("gelu_tanh", 8.0), ("gelu_tanh", 3.0)])
def test_sigmoid_forms(act, span, dtype):
    z = points(dtype, span)
    a, size, s, x = values(act, z.double())
    check(act_of(z, act), a, tolerance(act, dtype, a.abs(), x), z)
    check(slope_of(z, act), s, tolerance(act, dtype, size, x), z)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
def test_far_out(act, dtype):
    """Far out an activation is its argument or 0 (sigmoid: 1 or 0) and its slope 1 or 0 (sigmoid: 0); a NaN stays one."""
    top = 6e4 if dtype == torch.float16 else 3e38
    far = torch.tensor([200.0, 1e4, top] + ([] if dtype == torch.float16 else [1e10, 1e19, 1e20, 1e30])).to(dtype).cuda()
    one = torch.ones_like(far)
    assert torch.equal(act_of(far, act), one if act == "sigmoid" else far)
    assert torch.equal(act_of(-far, act), torch.zeros_like(far))
    assert torch.equal(slope_of(far, act), torch.zeros_like(far) if act == "sigmoid" else one)
    assert torch.equal(slope_of(-far, act), torch.zeros_like(far))
    nan = torch.full((3,), float("nan"), dtype=dtype, device="cuda")
    assert torch.isnan(act_of(nan, act)).all()
    if act != "relu":
        assert torch.isnan(slope_of(nan, act)).all()
