"""What training a classifier takes besides its layers, on CUDA tensors: layer norm (``layer_norm``), the embedding lookup
(``embedding``), each with its gradient, over the C entries of the same names. The package only marshals
arguments: every step runs in the kernels of ``libfusedxtx.so``.
"""
from __future__ import annotations

import torch

from ._lib import fxtx_embedding, fxtx_embedding_grad, fxtx_layer_norm, fxtx_layer_norm_grad
from .layers import _call, _current_stream, _features, _on_stream, _pitch, _type

_INT_BITS = {torch.int32: 32, torch.int64: 64}


def _vector(t, dtype, n, name, index):
    """The address of a contiguous n-vector, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} vector of length {n} on cuda:{index}")
    return t.data_ptr()


def _integers(t, m, name, index):
    """The address and the width of a contiguous vector of m int32 or int64 (m None: of any length)."""
    bits = _INT_BITS.get(t.dtype)
    if bits is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (int32 or int64)")
    if t.get_device() != index or t.dim() != 1 or (m is not None and t.shape[0] != m) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous vector of {'integers' if m is None else f'length {m}'} on cuda:{index}")
    return t.data_ptr(), bits


def layer_norm(X, weight=None, bias=None, eps: float = 1e-5, stats: bool = False, out=None, stream=None):
    """(X - mean) * rstd * weight + bias over each row of X (m, n), with rstd = (mean of (x - mean)^2 + eps)^-1/2.

    All tensors have one dtype (bfloat16, float16 or float32); sums are fp32 and results rounded once. ``weight`` and
    ``bias`` are (n,) or None; X and ``out`` are row-major, column slices of wider matrices included. ``stats=True``
    also returns mean and rstd, (m,) float32 tensors, as ``layer_norm_grad`` takes them. ``out`` may be X. Runs on the
    current stream, or on ``stream``, which then owns the new tensors. Autograd records nothing.
    """
    if stream is not None:
        context, stream = _on_stream(stream, X.get_device())
        with context:
            return layer_norm(X, weight, bias, eps, stats, out)
    code, dt, di, m, n, ldx = _features(X)
    pw, pb = _vector(weight, dt, n, "weight", di), _vector(bias, dt, n, "bias", di)
    if out is None:
        out, ldo = torch.empty((m, n), dtype=dt, device=X.device), n
    else:
        ldo = _pitch(out, dt, m, n, "out", di)
    mean = rstd = None
    if stats:
        mean, rstd = torch.empty((2, m), dtype=torch.float32, device=X.device).unbind()
    _call(fxtx_layer_norm, di, code, m, n, X.data_ptr(), ldx, pw, pb, eps, out.data_ptr(), ldo,
          mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None, _current_stream(di))
    return (out, mean, rstd) if stats else out


def layer_norm_grad(G, X, weight, mean, rstd, residual=None, need=(True, True, True), stream=None):
    """The gradient of ``layer_norm``: (dX, dweight, dbias) from the gradient ``G`` (m, n) at its result.

    With u = (X - mean) * rstd and h = G * weight, dX = rstd * (h - mean(h) - u * mean(h * u)) + residual, dweight = the
    column sums of G * u, dbias = those of G. ``residual`` (m, n) is the gradient that reaches X past the norm. ``need``
    says which of the three are computed; the others come back as None. Types, layouts and streams are those of
    ``layer_norm``.
    """
    if stream is not None:
        context, stream = _on_stream(stream, X.get_device())
        with context:
            return layer_norm_grad(G, X, weight, mean, rstd, residual, need)
    code, dt, di, m, n, ldx = _features(X)
    ldg = _pitch(G, dt, m, n, "G", di)
    pw = _vector(weight, dt, n, "weight", di)
    pm, ps = _vector(mean, torch.float32, m, "mean", di), _vector(rstd, torch.float32, m, "rstd", di)
    if pm is None or ps is None:
        raise ValueError("mean, rstd: the gradient needs the statistics that layer_norm kept")
    pr, ldr = None, 0
    if residual is not None:
        ldr, pr = _pitch(residual, dt, m, n, "residual", di), residual.data_ptr()
    want_x, want_w, want_b = need
    dX = torch.empty((m, n), dtype=dt, device=X.device) if want_x else None
    dw = torch.empty(n, dtype=dt, device=X.device) if want_w else None
    db = torch.empty(n, dtype=dt, device=X.device) if want_b else None
    _call(fxtx_layer_norm_grad, di, code, m, n, G.data_ptr(), ldg, X.data_ptr(), ldx, pw, pm, ps, pr, ldr,
          dX.data_ptr() if want_x else None, n, dw.data_ptr() if want_w else None, db.data_ptr() if want_b else None,
          _current_stream(di))
    return dX, dw, db


def embedding(ids, E, scale: float = 1.0, out=None, stream=None):
    """scale * E[ids]: rows of the table E (count, n) by ``ids`` (m,), int32 or int64, as an (m, n) tensor of E's dtype.

    An id outside 0 .. count - 1 stands for no row and gives zeros (-1 for padding). E and ``out`` are row-major,
    column slices included. Runs on the current stream, or on ``stream``, which then owns the new tensor.
    """
    if stream is not None:
        context, stream = _on_stream(stream, E.get_device())
        with context:
            return embedding(ids, E, scale, out)
    index, dt = E.get_device(), E.dtype
    if index < 0 or E.dim() != 2:
        raise ValueError("E: expected a 2-D CUDA tensor")
    code, (count, n) = _type(E, "E"), E.shape
    lde = _pitch(E, dt, count, n, "E", index)
    pi, bits = _integers(ids, None, "ids", index)
    m = ids.shape[0]
    if out is None:
        out, ldo = torch.empty((m, n), dtype=dt, device=E.device), n
    else:
        ldo = _pitch(out, dt, m, n, "out", index)
    _call(fxtx_embedding, index, code, m, n, count, pi, bits, E.data_ptr(), lde, scale, out.data_ptr(), ldo,
          _current_stream(index))
    return out


def embedding_grad(G, ids, count: int, scale: float = 1.0, out=None, stream=None):
    """The gradient of ``embedding``: row v of the (count, n) result is scale * the sum of the rows of G (m, n) whose id is v,
    zeros where there is none. Sums are fp32 and in a fixed order: the result is the same on every call. Every row of
    ``out`` is written. Ids and streams are those of ``embedding``.
    """
    if stream is not None:
        context, stream = _on_stream(stream, G.get_device())
        with context:
            return embedding_grad(G, ids, count, scale, out)
    index, dt = G.get_device(), G.dtype
    if index < 0 or G.dim() != 2:
        raise ValueError("G: expected a 2-D CUDA tensor")
    code, (m, n) = _type(G, "G"), G.shape
    ldg = _pitch(G, dt, m, n, "G", index)
    pi, bits = _integers(ids, m, "ids", index)
    if count < 0:
        raise ValueError("count: expected a number of rows")
    if out is None:
        out, ldo = torch.empty((count, n), dtype=dt, device=G.device), n
    else:
        ldo = _pitch(out, dt, count, n, "out", index)
    _call(fxtx_embedding_grad, index, code, m, n, count, G.data_ptr(), ldg, pi, bits, scale, out.data_ptr(), ldo,
          _current_stream(index))
    return out
