"""Sampling: the next tokens from rows of logits and given uniform numbers.

    sampler = Sampler(rows=64, vocab=163840)
    tokens, logprobs = sampler(logits, torch.rand(64, device="cuda"), temperature=0.7, top_p=0.9)

include/moe_serve.h states what the filters keep and which token is drawn.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import MoEError
from .serving import (LOGIT_DTYPES, SamplingStruct, StreamSpace, check, current_device, lib,
                      raw_stream, require, tensor)


class Sampler:
    """For calls of up to `rows` rows over a vocabulary of `vocab` tokens (at most
    2^19).  Calls run on the device's current stream and wait for nothing."""

    def __init__(self, rows: int, vocab: int, device="cuda"):
        for name, v in (("rows", rows), ("vocab", vocab)):
            require(isinstance(v, int) and 1 <= v < 1 << 31,
                    f"{name}: an integer from 1 on is needed, got {v!r}")
        self.rows, self.vocab, self._lib = rows, vocab, lib()
        w, c = ctypes.c_size_t(), ctypes.c_size_t()
        check(self._lib.moe_sample_workspace(rows, vocab, ctypes.byref(w), ctypes.byref(c)),
              "Sampler")
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.device, self._index = device, device.index
        self._space = StreamSpace(device, w.value, c.value)

    def _by_row(self, value, name, dtype, rows, off):
        """(address or None, the value for all rows)"""
        if value is None:
            return None, off
        if isinstance(value, torch.Tensor):
            tensor(value, name, dtype, (rows,), self.device)
            return value.data_ptr(), off
        if dtype == torch.int32:
            require(isinstance(value, int) and 0 <= value < 1 << 31,
                    f"{name}: an integer from 0 on is needed, got {value!r}")
        else:
            require(isinstance(value, (int, float)) and value >= 0 and math.isfinite(value),
                    f"{name}: a number from 0 on is needed, got {value!r}")
        return None, value

    def __call__(self, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
        """logits [rows, vocab] (bf16, fp16 or f32; rows contiguous), u [rows] f32 in
        [0, 1) (from 1 on: the last kept token).  temperature, top_p, min_p: numbers, or
        f32 tensors [rows]; top_k: an integer or an i32 tensor [rows]; None: 1, none,
        none, none.
        Temperature 0: the first largest logit.  Returns (tokens [rows] i32, the
        logarithms of the probabilities that they were drawn with [rows] f32); a
        row without anything above -inf gives -1 and -inf."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self(logits, u, temperature, top_k, top_p, min_p)
        if not isinstance(logits, torch.Tensor) or logits.dtype not in LOGIT_DTYPES or \
                logits.device != self.device:
            raise MoEError(f"logits: a bf16, fp16 or f32 tensor on {self.device} is needed")
        if logits.dim() != 2 or logits.shape[1] != self.vocab or logits.shape[0] > self.rows:
            raise MoEError(f"logits: shape {tuple(logits.shape)} given, (up to {self.rows}, "
                           f"{self.vocab}) needed")
        rows, (step, one) = logits.shape[0], logits.stride()
        if (one != 1 and self.vocab > 1) or (rows > 1 and step < self.vocab):
            raise MoEError(f"logits: strides {tuple(logits.stride())}: contiguous rows are needed")
        tensor(u, "u", torch.float32, (rows,), self.device)
        f32, by_row = torch.float32, self._by_row
        t, t_all = by_row(temperature, "temperature", f32, rows, 1.0)
        k, k_all = by_row(top_k, "top_k", torch.int32, rows, 0)
        p, p_all = by_row(top_p, "top_p", f32, rows, 1.0)
        m, m_all = by_row(min_p, "min_p", f32, rows, 0.0)
        tokens = torch.empty(rows, dtype=torch.int32, device=self.device)
        logprobs = torch.empty(rows, dtype=f32, device=self.device)
        if rows == 0:
            return tokens, logprobs
        stream = raw_stream(self._index)
        filters = SamplingStruct(t, p, m, k, t_all, p_all, m_all, k_all)
        with self._space.lock:
            w, c, _ = self._space.get(stream)
            check(self._lib.moe_sample(
                logits.data_ptr(), LOGIT_DTYPES[logits.dtype], step, rows, self.vocab, u.data_ptr(),
                ctypes.byref(filters), tokens.data_ptr(), logprobs.data_ptr(), w, c, stream), "sample")
        return tokens, logprobs
