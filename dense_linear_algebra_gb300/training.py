"""What training a classifier takes besides its layers, on CUDA tensors: layer norm (``layer_norm``), the embedding lookup
(``embedding``) and softmax cross entropy on a linear layer (``cross_entropy``), each with its gradient, over the C entries of the
same names. The package only marshals arguments: every step runs in the kernels of ``libfusedxtx.so``.
"""
from __future__ import annotations

import torch

from ._lib import (fxtx_cross_entropy, fxtx_cross_entropy_grad, fxtx_embedding, fxtx_embedding_grad, fxtx_layer_norm,
                   fxtx_layer_norm_grad)
from .layers import _call, _current_stream, _features, _on_stream, _pitch, _type, _weights

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
    mean = rstd = pm = ps = None
    if stats:
        mean, rstd = (torch.empty(m, dtype=torch.float32, device=X.device) for _ in range(2))
        pm, ps = mean.data_ptr(), rstd.data_ptr()
    _call(fxtx_layer_norm, di, code, m, n, X.data_ptr(), ldx, pw, pb, eps, out.data_ptr(), ldo, pm, ps, _current_stream(di))
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


def cross_entropy(X, W, labels, b=None, stream=None):
    """Softmax cross entropy on z = X W + b, without keeping z: (loss, lse), (m,) float32 tensors with lse_i = log sum_j exp z_ij
    and loss_i = lse_i - z_i,labels[i].

    X (m, n), W (n, k) and b (k,) have one dtype and are laid out as for ``linear``; n and k are at least 1. ``labels``:
    (m,), int32 or int64; a row whose label lies outside 0 .. k - 1 is left out (loss 0, no gradient). A bias of -inf
    takes a class out; a row without a class left has lse = -inf and a loss of NaN. Runs on the current stream, or on
    ``stream``, which then owns the new tensors. Autograd records nothing: ``cross_entropy_grad`` takes lse.
    """
    if stream is not None:
        context, stream = _on_stream(stream, X.get_device())
        with context:
            return cross_entropy(X, W, labels, b)
    code, dt, di, m, n, ldx = _features(X)
    k, ldw, trans = _weights(W, dt, n, di)
    pb = _vector(b, dt, k, "b", di)
    pl, bits = _integers(labels, m, "labels", di)
    loss, lse = (torch.empty(m, dtype=torch.float32, device=X.device) for _ in range(2))
    _call(fxtx_cross_entropy, di, code, m, n, k, X.data_ptr(), ldx, W.data_ptr(), ldw, trans, pb, pl, bits, loss.data_ptr(),
          lse.data_ptr(), _current_stream(di))
    return loss, lse


def cross_entropy_grad(X, W, labels, lse, b=None, g=1.0, need=(True, True, True), stream=None):
    """The gradient of ``cross_entropy``: with D_ij = g_i (exp(z_ij - lse_i) - [j = labels[i]]), (dX, dW, db) = (D W^T, X^T D, the
    column sums of D).

    ``g`` is the gradient at the losses: a number for all rows (1 / m for their mean), or an (m,) float32 tensor.
    ``need`` says which of the three are computed; the others come back as None. z is formed again, in pieces of the
    classes. D of a 16-bit type is rounded to it before the products; of float16 it is held multiplied by a power of two
    that brings the largest |g_i| of a row with a label to 2^14 .. 2^15, so that what is below 2^-39 of that is lost. db is
    summed from the unrounded values. dW is stored as W is: for W = P.t() it is the transposed view of a (k, n) tensor.
    Types, layouts, labels and streams are those of ``cross_entropy``.
    """
    if stream is not None:
        context, stream = _on_stream(stream, X.get_device())
        with context:
            return cross_entropy_grad(X, W, labels, lse, b, g, need)
    code, dt, di, m, n, ldx = _features(X)
    k, ldw, trans = _weights(W, dt, n, di)
    pb = _vector(b, dt, k, "b", di)
    pl, bits = _integers(labels, m, "labels", di)
    ps = _vector(lse, torch.float32, m, "lse", di)
    if ps is None:
        raise ValueError("lse: the gradient needs what cross_entropy gave")
    pg, gain = None, 1.0
    if isinstance(g, torch.Tensor):
        pg = _vector(g, torch.float32, m, "g", di)
    else:
        gain = float(g)
    device, (want_x, want_w, want_b) = X.device, need
    dX = torch.empty((m, n), dtype=dt, device=device) if want_x else None
    dW = torch.empty((k, n) if trans else (n, k), dtype=dt, device=device) if want_w else None
    db = torch.empty(k, dtype=dt, device=device) if want_b else None
    _call(fxtx_cross_entropy_grad, di, code, m, n, k, X.data_ptr(), ldx, W.data_ptr(), ldw, trans, pb, pl, bits, ps, pg, gain,
          dX.data_ptr() if want_x else None, n, dW.data_ptr() if want_w else None, n if trans else k,
          db.data_ptr() if want_b else None, _current_stream(di))
    return dX, dW.t() if trans and want_w else dW, db
