"""A paged key-value cache and the attention that reads it.

``PagedKV`` binds the tensors of a cache (the pages of every layer, the
sequences' page tables and lengths, the pages' reference counts) to the
library's operators on them:

  append   new keys and values into their pages (converted to e4m3 where the
           cache holds 8 bits)
  extend   longer sequences, and pages for them
  fork     copies of sequences that share their full pages
  free     sequences given up
  compact  the pages in use moved together

``PagedAttention`` plans attention over such a cache: ``decode`` for one new
token per sequence, ``prompt`` for many.  All of it runs on the cache's device,
on that device's current stream, reads lengths and tables on the device and
never waits for it, so calls can be captured into a HIP graph.
include/moe_serve.h states layouts and formulas.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import MoEError
from .serving import (DTYPES, AttnConfig, Cache, StreamSpace, check, current_device, lib,
                      raw_stream, require, tensor)

E4M3_MAX = 448.0
MAX_TOKENS = 1 << 24  # of a prompt call

# A kernel goes to the current device, and the default stream's handle, zero, is that
# of every device: each method that launches one makes its tensors' device current.


def _rows(t, name, heads, dim, dtypes, device) -> Tuple[int, int]:
    """Checks a [tokens][heads][dim] tensor whose rows are contiguous; returns
    its token and head strides (0 where there is only one, which may have any)."""
    # What is right is passed without forming any message: a call takes as long
    # as its smallest kernels.
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device:
        shape, (ts, hs, one) = t.shape, t.stride() if t.dim() == 3 else (0, 0, 0)
        if len(shape) == 3 and shape[1] == heads and shape[2] == dim and one == 1:
            if shape[0] <= 1:
                ts = 0
            if heads == 1:
                hs = 0
            if ts % 8 == 0 and hs % 8 == 0 and (heads == 1 or hs >= dim) and \
                    t.data_ptr() % 16 == 0:
                return ts, hs
    require(isinstance(t, torch.Tensor), f"{name}: a tensor is needed, got {type(t).__name__}")
    require(t.dtype in dtypes, f"{name}: {t.dtype} given, {' or '.join(map(str, dtypes))} needed")
    require(t.device == device, f"{name}: on {t.device}, not on {device}")
    shape, stride = t.shape, t.stride()
    require(len(shape) == 3 and shape[1] == heads and shape[2] == dim,
            f"{name}: shape {tuple(shape)} given, (tokens, {heads}, {dim}) needed")
    raise MoEError(f"{name}: strides {tuple(stride)}: rows of {dim} contiguous elements, 16-byte "
                   "aligned, are needed")


class PagedKV:
    """data [layers, 2, pages, kv_heads, page, head_dim] (bf16, fp16 or e4m3; keys
    at 0, values at 1), tables [seqs, cols] i32 (-1: no page), lengths [seqs]
    i32, refs [pages] i32; k_scale, v_scale [kv_heads] f32 for e4m3: a code c
    stands for c * scale.  The tensors stay the caller's and are changed in
    place; operations on them are ordered by the stream they run on.  The object
    (its flags, granted and scratch) is kept until its work on every stream is
    done."""

    def __init__(self, data, tables, lengths, refs, k_scale=None, v_scale=None):
        tensor(data, "data", tuple(DTYPES))
        require(data.dim() == 6 and data.shape[1] == 2,
                f"data: shape {tuple(data.shape)} given, (layers, 2, pages, kv_heads, page, "
                "head_dim) needed")
        dev = data.device
        layers, _, pages, heads, page, dim = data.shape
        tensor(tables, "tables", torch.int32, device=dev)
        require(tables.dim() == 2, f"tables: shape {tuple(tables.shape)} given, (seqs, cols) needed")
        seqs, cols = tables.shape
        tensor(lengths, "lengths", torch.int32, (seqs,), dev)
        tensor(refs, "refs", torch.int32, (pages,), dev)
        f8 = data.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                require(f8, f"{name}: only an e4m3 cache has scales")
                tensor(t, name, torch.float32, (heads,), dev)
        self.data, self.tables, self.lengths, self.refs = data, tables, lengths, refs
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device, self.dtype, self._index = dev, data.dtype, dev.index
        self.layers, self.pages, self.kv_heads, self.page, self.head_dim = \
            layers, pages, heads, page, dim
        self.seqs, self.cols = seqs, cols
        self.compute_dtypes = (torch.bfloat16, torch.float16) if f8 else (data.dtype,)
        self.flags = torch.zeros(1, dtype=torch.int32, device=dev)
        # positions that a sequence's last extend gave it (before any: no limit)
        self.granted = torch.full((seqs,), 2 ** 31 - 1, dtype=torch.int32, device=dev)
        self._granted_ptr = self.granted.data_ptr()
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.struct = Cache(data.data_ptr(), tables.data_ptr(), lengths.data_ptr(),
                            refs.data_ptr(), ptr(k_scale), ptr(v_scale), self.flags.data_ptr(),
                            DTYPES[data.dtype], layers, pages, heads, page, dim, seqs, cols)
        self._ref = ctypes.addressof(self.struct)
        self._lib = lib()
        check(self._lib.moe_kv_validate(self._ref), "PagedKV")
        size = self._lib.moe_kv_scratch_size(self._ref, seqs)
        self._scratch = torch.empty(size, dtype=torch.uint8, device=dev)
        self._scratch_ptr = self._scratch.data_ptr()

    @classmethod
    def empty(cls, layers, pages, kv_heads, page, head_dim, seqs, cols, dtype=torch.bfloat16,
              device="cuda", k_scale=None, v_scale=None) -> "PagedKV":
        """A new cache without sequences."""
        i32 = dict(dtype=torch.int32, device=device)
        data = torch.zeros((layers, 2, pages, kv_heads, page, head_dim), dtype=torch.uint8 if
                           dtype == torch.float8_e4m3fn else dtype, device=device).view(dtype)
        return cls(data, torch.full((seqs, cols), -1, **i32), torch.zeros(seqs, **i32),
                   torch.zeros(pages, **i32), k_scale, v_scale)

    def _list(self, t, name, n=None) -> int:
        tensor(t, name, torch.int32, None if n is None else (n,), self.device)
        if t.dim() != 1:
            raise MoEError(f"{name}: one dimension is needed")
        if t.shape[0] > self.seqs:
            raise MoEError(f"{name}: {t.shape[0]} entries for {self.seqs} sequences")
        return t.shape[0]

    def append(self, layer: int, k, v, cu=None, only_granted: bool = False) -> None:
        """Writes keys and values [tokens, kv_heads, head_dim] of new tokens,
        which the lengths count already.  cu None: token i is sequence i's last
        position (where it has none, nothing is written); else cu [batch + 1]
        i32: tokens cu[b] .. cu[b + 1] - 1 are sequence b's last positions.
        A sequence that extend could not lengthen has no new positions, and its
        tokens would go over its last ones, also in a full page that others
        share.  only_granted: nothing is written for a sequence with more
        tokens than its last extend gave it positions."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.append(layer, k, v, cu, only_granted)
        ts, hs = _rows(k, "k", self.kv_heads, self.head_dim, self.compute_dtypes, self.device)
        if _rows(v, "v", self.kv_heads, self.head_dim, (k.dtype,), self.device) != (ts, hs) or \
                v.shape != k.shape:
            raise MoEError("v: the shape and strides of k are needed")
        tokens = k.shape[0]
        if cu is None:
            batch = tokens
            if batch > self.seqs:
                raise MoEError(f"k: {batch} tokens for {self.seqs} sequences")
        else:
            tensor(cu, "cu", torch.int32, device=self.device)
            batch = cu.numel() - 1
            if cu.dim() != 1 or not 0 <= batch <= self.seqs:
                raise MoEError(f"cu: 1 to {self.seqs + 1} entries are needed, got shape "
                               f"{tuple(cu.shape)}")
        if not 0 <= layer < self.layers:
            raise MoEError(f"layer {layer} of {self.layers}")
        check(self._lib.moe_kv_append_granted(
            self._ref, layer, k.data_ptr(), v.data_ptr(), DTYPES[k.dtype], ts, hs, tokens,
            None if cu is None else cu.data_ptr(), batch,
            self._granted_ptr if only_granted else None, raw_stream(self._index)), "append")

    def free(self, seqs) -> None:
        """Gives up the (distinct) sequences of an i32 list."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.free(seqs)
        n = self._list(seqs, "seqs")
        check(self._lib.moe_kv_free(self._ref, seqs.data_ptr(), n, raw_stream(self._index)), "free")

    def fork(self, parents, children) -> None:
        """Sequence children[i], which holds nothing, becomes a copy of
        parents[i]: full pages are shared, a part-filled last page is copied."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.fork(parents, children)
        n = self._list(parents, "parents")
        self._list(children, "children", n)
        check(self._lib.moe_kv_fork(self._ref, parents.data_ptr(), children.data_ptr(), n,
                                    self._scratch_ptr, raw_stream(self._index)), "fork")

    def extend(self, counts, seqs=None) -> None:
        """Lengthens sequences (the first ones, or the distinct ones of the list
        seqs) by counts[i] positions, with pages for them.  One that pages or
        columns do not suffice for stays as it is; ``granted`` [seqs] holds what
        each sequence's last call gave it, counts[i] or 0."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.extend(counts, seqs)
        n = self._list(counts, "counts")
        if seqs is not None:
            self._list(seqs, "seqs", n)
        check(self._lib.moe_kv_extend_granted(
            self._ref, None if seqs is None else seqs.data_ptr(), counts.data_ptr(), n,
            self._granted_ptr, self._scratch_ptr, raw_stream(self._index)), "extend")

    def compact(self, out=None) -> None:
        """Moves the used pages to the front of the pool.  out (tables, refs):
        where the new tables and references go; None: into the cache's own."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.compact(out)
        tables, refs = out if out is not None else (self.tables, self.refs)
        if out is not None:
            tensor(tables, "out tables", torch.int32, (self.seqs, self.cols), self.device)
            tensor(refs, "out refs", torch.int32, (self.pages,), self.device)
        check(self._lib.moe_kv_compact(self._ref, tables.data_ptr(), refs.data_ptr(),
                                       self._scratch_ptr, raw_stream(self._index)), "compact")

    def read_flags(self) -> int:
        """Sticky flags (waits for the device): 1 fork or extend found too few
        free pages, 2 a sequence would have outgrown its table row."""
        return int(self.flags.item())


class PagedAttention:
    """Attention of q_heads query heads over a PagedKV, for calls of up to
    `batch` sequences.  longest: positions of the longest sequence to plan for;
    window and sinks: a row sees the last `window` positions up to its own and
    the first `sinks` (window 0: all up to its own); scale: of the scores,
    head_dim^-1/2 unless given."""

    def __init__(self, kv: PagedKV, q_heads: int, batch: int, longest: int, window: int = 0,
                 sinks: int = 0, scale: Optional[float] = None):
        self.kv, self.q_heads, self.batch = kv, q_heads, batch
        self.device, self._index = kv.device, kv.device.index
        # (The structure's 32 bits would take any integer, cut to them.)
        for name, v in (("q_heads", q_heads), ("batch", batch), ("longest", longest),
                        ("window", window), ("sinks", sinks)):
            require(isinstance(v, int) and 0 <= v < 1 << 31,
                    f"{name}: an integer from 0 to 2^31 - 1 is needed, got {v!r}")
        self.config = AttnConfig(q_heads, batch, longest, window, sinks,
                                 kv.head_dim ** -0.5 if scale is None else scale)
        self._cfg, self._lib = ctypes.addressof(self.config), lib()
        check(self._lib.moe_attn_validate(kv._ref, self._cfg), "PagedAttention")
        self._decode = self._space(0)
        self._prompt, self._prompt_tokens = None, 0

    def _space(self, tokens: int) -> StreamSpace:
        w, c = ctypes.c_size_t(), ctypes.c_size_t()
        check(self._lib.moe_attn_workspace(self.kv._ref, self._cfg, tokens, ctypes.byref(w),
                                           ctypes.byref(c)), "workspace")
        return StreamSpace(self.kv.device, w.value, c.value)

    def decode(self, layer: int, q):
        """q [batch, q_heads, head_dim], one new token of each of the first
        sequences, whose keys and values are in the cache.  Returns (out, like
        q; lse [batch, q_heads] f32)."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.decode(layer, q)
        kv = self.kv
        ts, hs = _rows(q, "q", self.q_heads, kv.head_dim, kv.compute_dtypes, kv.device)
        batch = q.shape[0]
        if not 1 <= batch <= self.batch:
            raise MoEError(f"q: {batch} sequences, planned for {self.batch}")
        if not 0 <= layer < kv.layers:
            raise MoEError(f"layer {layer} of {kv.layers}")
        out = torch.empty(q.shape, dtype=q.dtype, device=kv.device)
        lse = torch.empty((batch, self.q_heads), dtype=torch.float32, device=kv.device)
        stream = raw_stream(self._index)
        w, c, _ = self._decode.get(stream)
        check(self._lib.moe_attn_decode(kv._ref, self._cfg, layer, q.data_ptr(), DTYPES[q.dtype],
                                        ts, hs, batch, out.data_ptr(), lse.data_ptr(), w, c,
                                        stream), "decode")
        return out, lse

    def prompt(self, layer: int, q, cu, max_new: Optional[int] = None):
        """q [tokens, q_heads, head_dim]; cu [batch + 1] i32: rows cu[b] ..
        cu[b + 1] - 1 are the last positions of sequence b.  max_new: the most
        rows of one sequence, as other plans need it; this one reads cu, and
        answers do not depend on it.  Returns (out, like q; lse [tokens,
        q_heads] f32); rows that cu leaves out are not written."""
        if current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.prompt(layer, q, cu, max_new)
        kv = self.kv
        ts, hs = _rows(q, "q", self.q_heads, kv.head_dim, kv.compute_dtypes, kv.device)
        tensor(cu, "cu", torch.int32, device=kv.device)
        batch, tokens = cu.numel() - 1, q.shape[0]
        if cu.dim() != 1 or not 1 <= batch <= self.batch:
            raise MoEError(f"cu: {batch} sequences, planned for {self.batch}")
        if max_new is not None and not 0 <= max_new <= tokens:
            raise MoEError(f"max_new {max_new} of {tokens} tokens")
        if not 0 <= layer < kv.layers:
            raise MoEError(f"layer {layer} of {kv.layers}")
        out = torch.empty(q.shape, dtype=q.dtype, device=kv.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=kv.device)
        if tokens == 0:
            return out, lse
        stream = raw_stream(self._index)
        if tokens > self._prompt_tokens:
            # One space for all calls, of the largest one so far (what its work on a
            # stream still uses is not given to another stream before that is done).
            size = max(tokens, min(1 << (tokens - 1).bit_length(), MAX_TOKENS))
            self._prompt, self._prompt_tokens = self._space(size), size
        w, c, _ = self._prompt.get(stream)
        check(self._lib.moe_attn_prompt(kv._ref, self._cfg, layer, q.data_ptr(), DTYPES[q.dtype],
                                        ts, hs, tokens, cu.data_ptr(), batch, out.data_ptr(),
                                        lse.data_ptr(), w, c, stream), "prompt")
        return out, lse
