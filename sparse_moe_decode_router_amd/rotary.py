"""Rotary positions: which dimensions of a head are turned, and how fast.

``frequencies`` gives the usual geometric ones, stretched for long contexts or
not; ``Rotary`` keeps any on a device for ``PagedKV.append_rotated``.  Models differ in
how they stretch: one that does it in another way than ``frequencies`` says has its
own frequencies given to ``Rotary``.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import MoEError
from .serving import RotaryStruct, require


def frequencies(dim: int, base: float = 10000.0, factor: float = 1.0, original: int = 0,
                slow: float = 1.0, fast: float = 32.0) -> torch.Tensor:
    """[dim / 2] f64, in radians a position: base^(-2 j / dim).  factor: by how
    much a context longer than the `original` one stretches them.  Pairs that turn
    at least `fast` times within the original context stay, those that turn at most
    `slow` times are divided by the factor, and in between the frequency is a mean of
    the two in proportion to the turns (the pair's turns less `slow`, over `fast` less
    `slow`).  Others go in proportion to the pair's index between the two ends, which
    at slow 1 and fast 32 gives up to four times other frequencies: those are to be
    computed by the caller.  original 0: all are divided."""
    require(isinstance(dim, int) and dim > 0 and dim % 2 == 0, f"dim {dim!r}: an even number is needed")
    require(base > 0 and factor > 0 and original >= 0 and slow < fast,
            "base and factor above 0, an original context, and slow < fast are needed")
    j = torch.arange(dim // 2, dtype=torch.float64)
    f = base ** (-2 * j / dim)
    stay = torch.zeros_like(f)
    if original:
        stay = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
    return f * (stay + (1 - stay) / factor)


F32_MAX = torch.finfo(torch.float32).max


class Rotary:
    """frequencies [rot / 2]: radians a position of each pair.  The dimensions
    first .. first + rot - 1 of a head are turned (both multiples of 16), pair j
    of them being (2j, 2j + 1) if interleaved, else (j, j + rot / 2).  amplitude:
    what turned queries and keys are multiplied by.  Keep it as long as graphs that
    captured calls with it."""

    def __init__(self, frequencies, first: int = 0, interleaved: bool = False,
                 amplitude: float = 1.0, device="cuda"):
        f = torch.as_tensor(frequencies, dtype=torch.float64, device="cpu")
        require(f.dim() == 1 and f.numel() > 0 and f.numel() % 8 == 0,
                f"frequencies: shape {tuple(f.shape)} given, a multiple of 8 is needed")
        require(bool(f.isfinite().all()), "frequencies: finite ones are needed")
        require(isinstance(first, int) and first >= 0 and first % 16 == 0,
                f"first {first!r}: a multiple of 16 is needed")
        require(math.isfinite(amplitude) and abs(amplitude) <= F32_MAX,
                f"amplitude {amplitude!r}: a finite number of 32 bits is needed")
        self.turns = (f / (2 * math.pi)).to(device)
        self.device, self.first, self.rot = self.turns.device, first, 2 * f.numel()
        self.last = first + self.rot
        if self.last > 256:
            raise MoEError(f"dimensions up to {self.last}: heads have at most 256")
        self.interleaved, self.amplitude = bool(interleaved), float(amplitude)
        self.struct = RotaryStruct(self.turns.data_ptr(), first, self.rot, self.interleaved,
                                   self.amplitude)
        self._ref = ctypes.addressof(self.struct)
