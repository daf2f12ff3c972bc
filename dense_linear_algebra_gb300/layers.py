"""Layer operators on CUDA tensors: the fused linear layer (``linear``), its gradient (``linear_grad``) and the AdamW
step (``AdamW``), over the C entries ``fxtx_linear``, ``fxtx_linear_grad``, ``fxtx_adamw`` and ``fxtx_adamw_moments``.
The package only marshals arguments: every step runs in the kernels of ``libfusedxtx.so``.
"""
from __future__ import annotations

from array import array
from operator import attrgetter

import numpy as np
import torch

from . import _lib
from ._lib import _check, fxtx_adamw, fxtx_adamw_moments, fxtx_linear, fxtx_linear_grad

_current_device = torch.cuda.current_device
_current_stream = torch._C._cuda_getCurrentRawStream  # of a device, as the integer that the C entries take

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # fxtx_type_t

ADAMW_BLOCK = 256  # FXTX_ADAMW_BLOCK

_data_ptr, _numel, _get_device = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device
_is_contiguous, _dtype = torch.Tensor.is_contiguous, attrgetter("dtype")


def _type(t, name):
    code = TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return code


# fxtx_act_t
ACTS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "sigmoid": 5}


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act: expected one of {[a for a in ACTS if a]} or None, got {act!r}")
    return code


def _pitch(t, dtype, m, n, name, index):
    """The row pitch of a row-major (m, n) CUDA tensor."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (m, n):
        raise ValueError(f"{name}: expected a {dtype} matrix of shape {(m, n)} on cuda:{index}")
    if t.is_contiguous():
        return n
    ld, unit = t.stride()
    if m <= 1:
        ld = n
    if (unit != 1 and n > 1) or ld < n:
        raise ValueError(f"{name}: expected a row-major tensor with unit column stride")
    return ld


def _weights(W, dtype, n, index):
    """W (n, k): its columns' count, its pitch and whether it is stored by its columns."""
    if W.dtype is not dtype or W.get_device() != index or W.dim() != 2 or W.shape[0] != n:
        raise ValueError(f"W: expected a {dtype} matrix of {n} rows on cuda:{index}")
    k = W.shape[1]
    s0, s1 = W.stride()
    if (s1 == 1 or k <= 1) and (s0 >= k or n <= 1):
        return k, s0 if n > 1 else k, 0
    if (s0 == 1 or n <= 1) and (s1 >= n or k <= 1):
        return k, s1 if k > 1 else n, 1
    raise ValueError("W: expected unit stride along its rows or its columns")


def _features(X):
    """The type code, dtype, device, rows, features and row pitch of X."""
    index, dtype = X.get_device(), X.dtype
    if index < 0 or X.dim() != 2:
        raise ValueError("X: expected a 2-D CUDA tensor")
    m, n = X.shape
    return _type(X, "X"), dtype, index, m, n, _pitch(X, dtype, m, n, "X", index)


def _on_stream(stream, index):
    """The stream as a context that new tensors are made in, and as the C entries take it."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=index)
    return torch.cuda.stream(stream), stream.cuda_stream


def _call(fn, index, *args):
    """A C entry with the tensors' device current."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return _call(fn, index, *args)
    rc = fn(*args)
    if not rc:
        return
    if rc == _lib.FXTX_ERR_ALLOC and not torch.cuda.is_current_stream_capturing():
        # no argument has been written over that a second call reads: once more, with what torch caches given back
        torch.cuda.empty_cache()
        rc = fn(*args)
    if rc:
        _check(rc, fn.__name__)


def linear(X, W, b=None, act=None, residual=None, pre=False, out=None, stream=None):
    """act(X W + b) + residual in one pass: X (m, n), W (n, k), b (k), residual and the result (m, k).

    All tensors have one dtype (bfloat16, float16 or float32); sums are fp32 and rounded once. ``W`` may be a
    row-major (n, k) tensor or the transposed view of a row-major (k, n) one; the others are row-major, column slices
    of wider matrices included. ``act``: None, "relu", "gelu", "gelu_tanh", "silu" or "sigmoid". ``pre=True`` also
    returns Z = X W + b for ``linear_grad`` (or give the (m, k) tensor to keep it in). ``out`` may be ``residual``.
    Runs on the current stream, or on ``stream``, which then owns the new tensors.

    float32 values are taken as three bfloat16 terms each: an infinity comes out as a NaN (but for at most 16 rows of more
    than 64 features or outputs, 8 with W by columns, where it comes out as itself), and so may a value above 3.39e38.
    Nothing is recorded for autograd, whether or not a tensor requires a gradient: that is ``linear_grad``'s.
    """
    if stream is not None:
        context, stream = _on_stream(stream, X.get_device())
        with context:
            return linear(X, W, b, act, residual, pre, out)
    code, dt, di, m, n, ldx = _features(X)
    k, ldw, trans = _weights(W, dt, n, di)
    pb = pr = pz = None
    ldr = ldz = 0
    if b is not None:
        if b.dtype is not dt or b.get_device() != di or b.shape != (k,) or not b.is_contiguous():
            raise ValueError(f"b: expected a contiguous {dt} vector of length {k} on cuda:{di}")
        pb = b.data_ptr()
    if residual is not None:
        ldr, pr = _pitch(residual, dt, m, k, "residual", di), residual.data_ptr()
    if pre is True:
        pre, ldz = torch.empty((m, k), dtype=dt, device=X.device), k
        pz = pre.data_ptr()
    elif pre is not False and pre is not None:
        ldz, pz = _pitch(pre, dt, m, k, "pre", di), pre.data_ptr()
    else:
        pre = None
    if out is None:
        out, ldo = torch.empty((m, k), dtype=dt, device=X.device), k
    else:
        ldo = _pitch(out, dt, m, k, "out", di)
    _call(fxtx_linear, di, code, m, n, k, X.data_ptr(), ldx, W.data_ptr(), ldw, trans, pb, _act(act), pr, ldr, pz, ldz,
          out.data_ptr(), ldo, _current_stream(di))
    return out if pre is None else (out, pre)


def linear_grad(G, X, W, pre=None, act=None, need=(True, True, True), stream=None):
    """The gradient of ``linear``: with D = G * act'(pre), (dX, dW, db) = (D W^T, X^T D, the column sums of D).

    ``G`` (m, k) is the gradient at the result (and the gradient at the residual), ``pre`` the Z that ``linear`` kept
    (not needed without an activation). ``need`` says which of the three are computed; the others come back as None.
    Types, layouts and streams are those of ``linear``.

    D of a 16-bit type is rounded to it before the products, which doubles the squared error of bfloat16 results
    (2.35e-3 of the gradient, 1.66e-3 with D in fp32); in float16 it is 0 below 3e-8 and an infinity from 65,520 on. db
    is summed from D as it was.

    dW is stored as W is: for W = P.t() it is the transposed view of a (k, n) tensor, and ``dW.t()`` is the contiguous
    gradient of P that ``AdamW.step`` takes.
    """
    if stream is not None:
        context, stream = _on_stream(stream, X.get_device())
        with context:
            return linear_grad(G, X, W, pre, act, need)
    code, dt, di, m, n, ldx = _features(X)
    kind = _act(act)
    k, ldw, trans = _weights(W, dt, n, di)
    ldg = _pitch(G, dt, m, k, "G", di)
    pz, ldz = None, 0
    if kind:
        if pre is None:
            raise ValueError("pre: the gradient of an activation needs the Z that linear kept")
        ldz, pz = _pitch(pre, dt, m, k, "pre", di), pre.data_ptr()
    device, (want_x, want_w, want_b) = X.device, need
    dX = dW = db = px = pw = pb = None
    if want_x:
        dX = torch.empty((m, n), dtype=dt, device=device)
        px = dX.data_ptr()
    if want_w:
        dW = torch.empty((k, n) if trans else (n, k), dtype=dt, device=device)
        pw = dW.data_ptr()
    if want_b:
        db = torch.empty(k, dtype=dt, device=device)
        pb = db.data_ptr()
    _call(fxtx_linear_grad, di, code, m, n, k, G.data_ptr(), ldg, X.data_ptr(), ldx, W.data_ptr(), ldw, trans, pz, ldz,
          kind, px, n, pw, n if trans else k, pb, _current_stream(di))
    return dX, dW.t() if trans and want_w else dW, db


class AdamW:
    """AdamW over a list of tensors, all updated in one launch a step.

        m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
        p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)

    ``params``: contiguous CUDA tensors of one dtype (float32, bfloat16 or float16) on one device, not overlapping;
    they are updated in place. ``copies``: None, or tensors of the params' sizes and one dtype that receive the new
    values too (a bfloat16 working copy of float32 weights). Arithmetic is fp32 whatever the types.

    ``state_bits`` 32 holds both moments in fp32 (8 bytes an element). 8 holds each in one byte with an fp32 scale for
    every 256 elements of a tensor: the first moment as ``scale * c * |c|`` with int8 ``c``, the second as its root
    ``scale * c * c`` with uint8 ``c``, rounded to nearest (a change smaller than half a step of the code is lost; an
    infinity or a NaN in a gradient makes its block's moments NaN, and a gradient whose square is above fp32's range
    its block's second moments: the block's params are NaN from the next step on).

    The states of all tensors lie one after the other in flat tensors, each starting at a multiple of 256 elements
    (``offsets``): ``exp_avg`` and ``exp_avg_sq``, and for 8 bits ``exp_avg_scale`` and ``exp_avg_sq_scale``.
    ``steps`` counts the steps taken; ``lr`` and the other settings may be changed between steps. A step that a CUDA graph
    captured is replayed with the step number and settings of its capture.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, copies=None):
        self.params = list(params)
        if not self.params:
            raise ValueError("params: an empty list")
        if state_bits not in (8, 32):
            raise ValueError("state_bits: expected 8 or 32")
        first = self.params[0]
        if not first.is_cuda:
            raise ValueError("params: expected CUDA tensors")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.steps = state_bits, 0
        self._device, self._index = first.device, first.get_device()
        self._dtype, self._type = first.dtype, _type(first, "params")
        self._sizes = [p.numel() for p in self.params]
        self.copies = None if copies is None else list(copies)
        self._copy_type = 0 if self.copies is None else _type(self.copies[0], "copies")
        self._copy_dtype = None if self.copies is None else self.copies[0].dtype
        at = np.zeros(len(self._sizes) + 1, dtype=np.int64)
        np.cumsum([(n + ADAMW_BLOCK - 1) // ADAMW_BLOCK for n in self._sizes], out=at[1:])
        self.offsets = [int(b) * ADAMW_BLOCK for b in at[:-1]]
        blocks = int(at[-1])
        self._total = total = blocks * ADAMW_BLOCK
        wide = state_bits == 32
        self._m = torch.zeros(total, dtype=torch.float32 if wide else torch.int8, device=self._device)
        self._v = torch.zeros(total, dtype=torch.float32 if wide else torch.uint8, device=self._device)
        self._ms = self._vs = None
        # the kernel's table, one fxtx_adamw_tensor_t a tensor: n, p, g, m, v, m_scale, v_scale, copy
        table = np.zeros((len(self._sizes), 8), dtype=np.int64)
        start = at[:-1] * ADAMW_BLOCK * (4 if wide else 1)
        table[:, 3] = self._m.data_ptr() + start
        table[:, 4] = self._v.data_ptr() + start
        if not wide:
            self._ms = torch.zeros(blocks, dtype=torch.float32, device=self._device)
            self._vs = torch.zeros(blocks, dtype=torch.float32, device=self._device)
            table[:, 5] = self._ms.data_ptr() + at[:-1] * 4
            table[:, 6] = self._vs.data_ptr() + at[:-1] * 4
        self._table = array("q", table.tobytes())
        self._where = self._copy_where = None
        self._hold()

    exp_avg = property(lambda self: self._m)
    exp_avg_sq = property(lambda self: self._v)
    exp_avg_scale = property(lambda self: self._ms)
    exp_avg_sq_scale = property(lambda self: self._vs)

    def _hold(self):
        """Takes the params' (and copies') addresses into the table, holding on to their memory: an address seen
        again then stands for the same memory, and needs no other check."""
        self._where = self._pointers(self.params, self._dtype, "params")
        self._held = [p.detach() for p in self.params]
        self._table[1::8] = array("q", self._where)
        if self.copies is not None:
            self._copy_where = self._pointers(self.copies, self._copy_dtype, "copies")
            self._held += [c.detach() for c in self.copies]
            self._table[7::8] = array("q", self._copy_where)

    def _pointers(self, tensors, dtype, name, optional=False):
        """The tensors' addresses (0 for a None where that is allowed), each checked against the size that the states
        were made for."""
        try:  # one pass a property, none of it interpreted a tensor at a time
            if (list(map(_numel, tensors)) == self._sizes and set(map(_dtype, tensors)) == {dtype}
                    and set(map(_get_device, tensors)) == {self._index} and all(map(_is_contiguous, tensors))):
                return list(map(_data_ptr, tensors))
        except (TypeError, AttributeError):  # a None, or no tensor
            pass
        if len(tensors) != len(self._sizes):
            raise ValueError(f"{name}: expected {len(self._sizes)} tensors, got {len(tensors)}")
        index, got = self._index, []
        for t, n in zip(tensors, self._sizes):
            if t is None and optional:
                got.append(0)
                continue
            if t is None or t.dtype is not dtype or t.numel() != n or t.get_device() != index or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous {dtype} tensors of the params' sizes on cuda:{index}")
            got.append(t.data_ptr())
        return got

    def step(self, grads, stream=None) -> None:
        """Updates the params (and copies) from ``grads``: contiguous tensors of the params' sizes and one dtype. A
        gradient may be None: its tensor and moments stay as they are. Asynchronous on the current stream (or
        ``stream``)."""
        grads = list(grads)
        kind = next((g for g in grads if g is not None), None)
        if kind is None:
            raise ValueError("grads: no gradient")
        g_type = _type(kind, "grads")
        if list(map(_data_ptr, self.params)) != self._where or (
                self.copies is not None and list(map(_data_ptr, self.copies)) != self._copy_where):
            self._hold()
        table, where = self._table, self._pointers(grads, kind.dtype, "grads", optional=True)
        table[2::8] = array("q", where)
        # an entry of no elements is left out
        table[0::8] = array("q", [n if g else 0 for g, n in zip(where, self._sizes)] if 0 in where else self._sizes)
        _call(fxtx_adamw, self._index, len(where), table.buffer_info()[0], self._type, g_type, self._copy_type,
              self.state_bits, self.steps + 1, self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
              _current_stream(self._index) if stream is None else
              stream if isinstance(stream, int) else stream.cuda_stream)
        self.steps += 1

    def moments(self, stream=None):
        """Both moments of all tensors as flat fp32 tensors (laid out by ``offsets``): the states themselves for 32
        bits, for 8 the values that they stand for."""
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        if stream is not None:
            context, stream = _on_stream(stream, self._index)
            with context:
                return self.moments()
        m = torch.empty(self._total, dtype=torch.float32, device=self._device)
        v = torch.empty(self._total, dtype=torch.float32, device=self._device)
        _call(fxtx_adamw_moments, self._index, self._total, self.exp_avg.data_ptr(), self.exp_avg_scale.data_ptr(),
              self.exp_avg_sq.data_ptr(), self.exp_avg_sq_scale.data_ptr(), m.data_ptr(), v.data_ptr(),
              _current_stream(self._index))
        return m, v

    def _state(self):
        names = ["exp_avg", "exp_avg_sq"] + (["exp_avg_scale", "exp_avg_sq_scale"] if self.state_bits == 8 else [])
        return {name: getattr(self, name) for name in names}

    def state_dict(self) -> dict:
        """The step count, the tensors' sizes and copies of the held states (codes and scales for 8 bits)."""
        return {"steps": self.steps, "sizes": list(self._sizes)} | {name: t.clone() for name, t in self._state().items()}

    def load_state_dict(self, state: dict) -> None:
        """Takes over what ``state_dict`` gave for tensors of the same sizes and the same ``state_bits``. A state put together
        by other means may leave ``sizes`` out: its tensors are then laid out by ``offsets``."""
        held = self._state()
        for name, t in held.items():
            if name not in state or state[name].dtype is not t.dtype or state[name].shape != t.shape:
                raise ValueError(f"{name}: expected a {t.dtype} tensor of {t.numel()} elements")
        if "sizes" in state and list(state["sizes"]) != self._sizes:
            raise ValueError("sizes: the state is of other tensors, or of these in another order")
        if "steps" not in state:
            raise ValueError("steps: missing")
        steps = int(state["steps"])
        for name, t in held.items():
            t.copy_(state[name])
        self.steps = steps
