"""Linear layer of a decode batch with its epilogue: torch layer over
alspec_linear."""
from __future__ import annotations

import torch

from . import alspec as _c
from .alspec import AlspecError
from .paged import _CODES, _FLOATS, _empty, _on, _settle, _stream, _take_error, _want


class Linear:
    """y = activation(x W^T + bias) + residual, bf16 x and W, fp32 sums.

    ``weight`` is bf16 [n, k] contiguous (k a multiple of 8), ``bias`` bf16 [n]
    or None, ``activation`` "none", "relu", "gelu" (erf) or "silu".
    """

    def __init__(self, weight, bias=None, activation="none"):
        _want(weight.dim() == 2 and weight.dtype is torch.bfloat16 and weight.is_cuda
              and weight.is_contiguous() and weight.shape[0] > 0 and weight.shape[1] > 0
              and weight.shape[1] % 8 == 0,
              "weight: a contiguous bf16 CUDA tensor [n, k] with k a multiple of 8 is needed")
        _want(bias is None or (tuple(bias.shape) == (weight.shape[0],)
                               and bias.dtype is torch.bfloat16 and bias.device == weight.device
                               and bias.is_contiguous()),
              "bias: a contiguous bf16 tensor [n] on the weight's device is needed")
        _want(activation in _c.ACTIVATIONS,
              f"activation {activation!r}: one of {sorted(_c.ACTIVATIONS)} is needed")
        self.weight, self.bias, self.device = weight, bias, weight.device
        self.n, self.k = weight.shape
        self.activation = _c.ACTIVATIONS[activation]
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._index = self.device.index
        _settle(self.device)

    def apply(self, x, residual=None, out=None, out_dtype=torch.bfloat16, stream=None):
        """x bf16 [rows, k] (rows may be slices of wider ones); residual, if
        given, and out are contiguous [rows, n] tensors of one type (fp32 or
        bf16) and may be the same tensor; out overlaps nothing else that is
        read.  Returns out; a new one has the residual's type, without a
        residual ``out_dtype``, and belongs to the stream of the call."""
        dev, n = self.device, self.n
        rows = x.shape[0]
        xt = x.stride()
        if not (x.shape == (rows, self.k) and x.dtype is torch.bfloat16 and x.device == dev
                and xt[1] == 1 and (rows <= 1 or xt[0] > 0)):
            raise ValueError(f"x: a bf16 tensor [rows, {self.k}] on {dev} with consecutive "
                             f"columns and rows not broadcast is needed, got {x.dtype} "
                             f"{tuple(x.shape)} on {x.device}")
        if out is None:
            out = _empty((rows, n), out_dtype if residual is None else residual.dtype, dev,
                         stream)
        if not (out.shape == (rows, n) and out.dtype in _FLOATS and out.device == dev
                and out.is_contiguous()):
            raise ValueError(f"out: a contiguous tensor [{rows}, {n}] in fp32 or bf16 on {dev} "
                             f"is needed, got {out.dtype} {tuple(out.shape)} on {out.device}")
        if residual is not None and not (residual.shape == (rows, n)
                                         and residual.dtype is out.dtype
                                         and residual.device == dev
                                         and residual.is_contiguous()):
            raise ValueError(f"residual: a contiguous tensor [{rows}, {n}] of out's type "
                             f"{out.dtype} on {dev} is needed, got {residual.dtype} "
                             f"{tuple(residual.shape)} on {residual.device}")
        st = _on(self._index, _c._lib.alspec_linear, x.data_ptr(), 0 if rows <= 1 else xt[0],
                 self.weight.data_ptr(), 0 if self.bias is None else self.bias.data_ptr(),
                 0 if residual is None else residual.data_ptr(), out.data_ptr(),
                 _CODES[out.dtype], self.activation, rows, n, self.k, self.err.data_ptr(),
                 _stream(stream, self._index))
        if st:
            raise AlspecError(st, "alspec_linear")
        return out

    def device_error(self, stream=None):
        """(status, error word), read and cleared; synchronizes the stream."""
        return _take_error(self.err, _c.ALSPEC_ERR_TIMEOUT, stream, self.device)
