"""Products with 4-bit weights: y = x W^T, W = (codes - zeros) * scales.

codes [n, k / 2] u8 hold two columns per byte (2j in the low half), scales
[n, k / group] one factor per group of 32, 64 or 128 columns in x's type, zeros
[n, k / group] u8 the code that stands for zero (None: 8).
"""
from __future__ import annotations

import torch

from .binding import MoEError
from .serving import DTYPES, check, current_device, lib, raw_stream, require, tensor

GROUPS = (32, 64, 128)


class W4Linear:
    """A linear layer over 4-bit weights; the tensors are kept as they are."""

    def __init__(self, codes, scales, zeros=None):
        tensor(codes, "codes", torch.uint8)
        require(codes.dim() == 2, f"codes: shape {tuple(codes.shape)} given, (n, k / 2) needed")
        dev = codes.device
        tensor(scales, "scales", (torch.bfloat16, torch.float16), device=dev)
        self.n, self.k = codes.shape[0], 2 * codes.shape[1]
        require(scales.dim() == 2 and scales.shape[0] == self.n and scales.shape[1] > 0 and
                self.k % scales.shape[1] == 0 and self.k // scales.shape[1] in GROUPS,
                f"scales: shape {tuple(scales.shape)} for {self.n} rows of {self.k} columns: "
                "(n, k / group) with groups of 32, 64 or 128 needed")
        self.group = self.k // scales.shape[1]
        if zeros is not None:
            tensor(zeros, "zeros", torch.uint8, scales.shape, dev)
        self.codes, self.scales, self.zeros = codes, scales, zeros
        self.device, self._index, self.dtype = dev, dev.index, scales.dtype
        self._lib, self._dtype = lib(), DTYPES[self.dtype]
        self._ptrs = (codes.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None
                      else None)

    def __call__(self, x, out=None):
        """x [tokens, k], rows contiguous -> [tokens, n]."""
        if current_device() != self._index:  # kernels go to the current device
            with torch.cuda.device(self.device):
                return self(x, out)
        if not isinstance(x, torch.Tensor) or x.dtype != self.dtype or x.device != self.device:
            raise MoEError(f"x: a {self.dtype} tensor on {self.device} is needed")
        shape, stride = x.shape, x.stride()
        if len(shape) != 2 or shape[1] != self.k:
            raise MoEError(f"x: shape {tuple(shape)} given, (tokens, {self.k}) needed")
        address, tokens = x.data_ptr(), shape[0]
        step = stride[0] if tokens > 1 else 0  # (that of a single row may be any)
        if stride[1] != 1 or step % 8 or address % 16:
            raise MoEError(f"x: strides {tuple(stride)}: contiguous rows, 16-byte aligned, are "
                           "needed")
        if out is None:
            out = torch.empty((tokens, self.n), dtype=x.dtype, device=self.device)
        else:
            tensor(out, "out", x.dtype, (tokens, self.n), self.device)
        codes, scales, zeros = self._ptrs
        check(self._lib.moe_w4_linear(address, step, self._dtype, codes, scales,
                                      zeros, tokens, self.k, self.n, self.group, out.data_ptr(),
                                      raw_stream(self._index)), "w4")
        return out
