"""Linear layer of a decode batch with its epilogue: torch layer over
alspec_linear."""
from __future__ import annotations

import torch

from . import alspec as _c
from .alspec import AlspecError
from .paged import _On, _stream, _want


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
        with _On(self.device):
            self.err = torch.zeros(1, dtype=torch.int32, device=self.device)

    def apply(self, x, residual=None, out=None, out_dtype=torch.bfloat16, stream=None):
        """x bf16 [rows, k] (rows may be slices of wider ones); residual, if
        given, and out are contiguous [rows, n] tensors of one type (fp32 or
        bf16; ``out_dtype`` where out is to be made) and may be the same
        tensor.  Returns out."""
        dev = self.device
        rows = x.shape[0]
        _want(x.dim() == 2 and x.shape[1] == self.k and x.dtype is torch.bfloat16
              and x.device == dev and x.stride(1) == 1,
              f"x: a bf16 tensor [rows, {self.k}] on {dev} with consecutive columns is needed")
        if out is None:
            out = torch.empty((rows, self.n), device=dev,
                              dtype=out_dtype if residual is None else residual.dtype)
        for name, t in (("out", out), ("residual", residual)):
            _want(t is None or (tuple(t.shape) == (rows, self.n) and t.device == dev
                                and t.dtype in (torch.float32, torch.bfloat16)
                                and t.dtype is out.dtype and t.is_contiguous()),
                  f"{name}: a contiguous tensor [{rows}, {self.n}] in fp32 or bf16 (out's type) "
                  f"on {dev} is needed")
        with _On(dev):
            st = _c.alspec_linear(
                x.data_ptr(), 0 if rows <= 1 else x.stride(0), self.weight.data_ptr(),
                0 if self.bias is None else self.bias.data_ptr(),
                0 if residual is None else residual.data_ptr(), out.data_ptr(),
                _c.ALSPEC_F32 if out.dtype is torch.float32 else _c.ALSPEC_BF16,
                self.activation, rows, self.n, self.k, self.err.data_ptr(),
                _stream(stream, dev))
        if st:
            raise AlspecError(st, "alspec_linear")
        return out

    def device_error(self, stream=None):
        """(status, error word), read and cleared; synchronizes the stream."""
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        with _On(self.device), torch.cuda.stream(s):
            word = int(self.err.item())
            self.err.zero_()
        return (_c.ALSPEC_ERR_TIMEOUT if word else _c.ALSPEC_OK), word
