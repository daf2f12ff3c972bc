"""Layer operators on CUDA tensors: the AdamW step (``AdamW``) over the C entries ``fxtx_adamw`` and
``fxtx_adamw_moments``. The package only marshals arguments: every step runs in the kernels of ``libfusedxtx.so``.
"""
from __future__ import annotations

import numpy as np
import torch

from . import _lib
from ._lib import _check, _on, _stream

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # fxtx_type_t

ADAMW_BLOCK = 256  # FXTX_ADAMW_BLOCK


def _type(t, name):
    code = TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return code


class AdamW:
    """AdamW over a list of tensors, all updated in one launch a step.

        m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
        p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)

    ``params``: contiguous CUDA tensors of one dtype (float32, bfloat16 or float16) on one device, not overlapping;
    they are updated in place. ``copies``: None, or tensors of the params' sizes and one dtype that receive the new
    values too (a bfloat16 working copy of float32 weights). Arithmetic is fp32 whatever the types.

    ``state_bits`` 32 holds both moments in fp32 (8 bytes an element). 8 holds each in one byte with an fp32 scale for
    every 256 elements of a tensor: the first moment as ``scale * c * |c|`` with int8 ``c``, the second as its root
    ``scale * c * c`` with uint8 ``c``, rounded to nearest (a change smaller than half a step of the code is lost, and
    an infinity or a NaN in a gradient makes its block's moments NaN).

    The states of all tensors lie one after the other in flat tensors, each starting at a multiple of 256 elements
    (``offsets``): ``exp_avg`` and ``exp_avg_sq``, and for 8 bits ``exp_avg_scale`` and ``exp_avg_sq_scale``.
    ``steps`` counts the steps taken; ``lr`` and the other settings may be changed between steps.
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
        # the kernel's table (fxtx_adamw_tensor_t): n, p, g, m, v, m_scale, v_scale, copy
        self._table = np.zeros((len(self._sizes), 8), dtype=np.int64)
        self._table[:, 0] = self._sizes
        wide = state_bits == 32
        self.exp_avg = torch.zeros(total, dtype=torch.float32 if wide else torch.int8, device=self._device)
        self.exp_avg_sq = torch.zeros(total, dtype=torch.float32 if wide else torch.uint8, device=self._device)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        start = at[:-1] * ADAMW_BLOCK * (4 if wide else 1)
        self._table[:, 3] = self.exp_avg.data_ptr() + start
        self._table[:, 4] = self.exp_avg_sq.data_ptr() + start
        if not wide:
            self.exp_avg_scale = torch.zeros(blocks, dtype=torch.float32, device=self._device)
            self.exp_avg_sq_scale = torch.zeros(blocks, dtype=torch.float32, device=self._device)
            self._table[:, 5] = self.exp_avg_scale.data_ptr() + at[:-1] * 4
            self._table[:, 6] = self.exp_avg_sq_scale.data_ptr() + at[:-1] * 4
        self._pointers(self.params, self._dtype, "params")
        if self.copies is not None:
            self._pointers(self.copies, self._copy_dtype, "copies")

    def _pointers(self, tensors, dtype, name, optional=False):
        """The tensors' addresses (0 for a None where that is allowed), each checked against the size that the states
        were made for."""
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
        table = self._table
        table[:, 1] = self._pointers(self.params, self._dtype, "params")
        table[:, 2] = self._pointers(grads, kind.dtype, "grads", optional=True)
        if self.copies is not None:
            table[:, 7] = self._pointers(self.copies, self._copy_dtype, "copies")
        # an entry of no elements is left out
        table[:, 0] = [0 if g is None else n for g, n in zip(grads, self._sizes)]
        with _on(self._index):
            rc = _lib.fxtx_adamw(len(self._sizes), table.ctypes.data, self._type, g_type, self._copy_type,
                                 self.state_bits, self.steps + 1, self.lr, self.betas[0], self.betas[1], self.eps,
                                 self.weight_decay, _stream(stream, self._device))
        _check(rc, "fxtx_adamw")
        self.steps += 1

    def moments(self, stream=None):
        """Both moments of all tensors as flat fp32 tensors (laid out by ``offsets``): the states themselves for 32
        bits, for 8 the values that they stand for."""
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        m = torch.empty(self._total, dtype=torch.float32, device=self._device)
        v = torch.empty(self._total, dtype=torch.float32, device=self._device)
        with _on(self._index):
            rc = _lib.fxtx_adamw_moments(self._total, self.exp_avg.data_ptr(), self.exp_avg_scale.data_ptr(),
                                         self.exp_avg_sq.data_ptr(), self.exp_avg_sq_scale.data_ptr(), m.data_ptr(),
                                         v.data_ptr(), _stream(stream, self._device))
        _check(rc, "fxtx_adamw_moments")
        return m, v

    def _state(self):
        names = ["exp_avg", "exp_avg_sq"] + (["exp_avg_scale", "exp_avg_sq_scale"] if self.state_bits == 8 else [])
        return {name: getattr(self, name) for name in names}

    def state_dict(self) -> dict:
        """The step count and copies of the held states (codes and scales for 8 bits)."""
        return {"steps": self.steps} | {name: t.clone() for name, t in self._state().items()}

    def load_state_dict(self, state: dict) -> None:
        """Takes over what ``state_dict`` gave for tensors of the same sizes and the same ``state_bits``."""
        held = self._state()
        for name, t in held.items():
            if name not in state or state[name].dtype is not t.dtype or state[name].shape != t.shape:
                raise ValueError(f"{name}: expected a {t.dtype} tensor of {t.numel()} elements")
        for name, t in held.items():
            t.copy_(state[name])
        self.steps = int(state["steps"])
