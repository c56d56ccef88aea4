"""Loading of ``libmoe_serve.so`` (the C ABI in include/moe_serve.h) and what
the modules above it (``attention``, ``w4``) share: the argument structures,
dtype codes, checks of tensors and the status codes.

Argument marshalling only, as in ``binding``: the operators run in the HIP
kernels of the library, and there is nothing to fall back to.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .binding import MOE_ERR_HIP, MOE_OK, MoEError

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_serve.so")

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}
STATUS = {-1: "invalid argument", -2: "unsupported shape or device", -3: "HIP error",
          -4: "workspace missing, too small or misaligned"}
EXPORTED = ("moe_kv_validate", "moe_kv_append", "moe_kv_append_granted", "moe_kv_free",
            "moe_kv_scratch_size", "moe_kv_fork", "moe_kv_extend", "moe_kv_extend_granted",
            "moe_kv_compact", "moe_attn_validate", "moe_attn_workspace", "moe_attn_decode",
            "moe_attn_prompt", "moe_w4_linear", "moe_serve_last_hip_error")

_lib = None


class Cache(ctypes.Structure):
    """moe_kv_cache"""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("data", "tables", "lengths", "refs", "k_scale", "v_scale", "flags")] + \
               [(n, ctypes.c_int32) for n in
                ("dtype", "layers", "pages", "kv_heads", "page", "head_dim", "seqs", "cols")]


class AttnConfig(ctypes.Structure):
    """moe_attn_config"""
    _fields_ = [(n, ctypes.c_int32) for n in ("q_heads", "batch", "longest", "window", "sinks")] + \
               [("scale", ctypes.c_float)]


def lib() -> ctypes.CDLL:
    """Loads the library (it must have been built: __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MoEError(f"{LIB_PATH} is missing: build the HIP library first "
                       "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sizes = [ctypes.POINTER(size), ctypes.POINTER(size)]
    args = {
        "moe_kv_validate": [vp],
        "moe_kv_append": [vp, i32, vp, vp, i32, i64, i64, i32, vp, i32, vp],
        "moe_kv_append_granted": [vp, i32, vp, vp, i32, i64, i64, i32, vp, i32, vp, vp],
        "moe_kv_free": [vp, vp, i32, vp],
        "moe_kv_scratch_size": [vp, i32],
        "moe_kv_fork": [vp, vp, vp, i32, vp, vp],
        "moe_kv_extend": [vp, vp, vp, i32, vp, vp],
        "moe_kv_extend_granted": [vp, vp, vp, i32, vp, vp, vp],
        "moe_kv_compact": [vp, vp, vp, vp, vp],
        "moe_attn_validate": [vp, vp],
        "moe_attn_workspace": [vp, vp, i32] + sizes,
        "moe_attn_decode": [vp, vp, i32, vp, i32, i64, i64, i32, vp, vp, vp, vp, vp],
        "moe_attn_prompt": [vp, vp, i32, vp, i32, i64, i64, i32, vp, i32, vp, vp, vp, vp, vp],
        "moe_w4_linear": [vp, i64, i32, vp, vp, vp, i32, i32, i32, i32, vp, vp],
        "moe_serve_last_hip_error": [],
    }
    for name in EXPORTED:
        f = getattr(L, name)
        f.argtypes = args[name]
        f.restype = size if name == "moe_kv_scratch_size" else i32
    _lib = L
    return L


def check(rc: int, what: str) -> None:
    if rc != MOE_OK:
        extra = ""
        if rc == MOE_ERR_HIP:
            extra = f" (hip error {lib().moe_serve_last_hip_error()})"
        raise MoEError(f"{what}: {STATUS.get(rc, 'error')}{extra} [{rc}]")


# By a device's index: the handle of its current stream; and the current device.
# (Without the Python objects in between, where this torch has it: a call of a few
# microseconds notices the difference.)
raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                     lambda index: torch.cuda.current_stream(index).cuda_stream)
current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def require(cond: bool, message: str) -> None:
    if not cond:
        raise MoEError(message)


def tensor(t, name: str, dtype, shape=None, device=None) -> torch.Tensor:
    """A contiguous GPU tensor of that type (and shape, and device), or MoEError."""
    # (What is right is passed without forming any message.)
    if isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and \
            (t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype) and \
            (shape is None or tuple(t.shape) == tuple(shape)) and \
            (device is None or t.device == device):
        return t
    require(isinstance(t, torch.Tensor), f"{name}: a tensor is needed, got {type(t).__name__}")
    require(t.is_cuda, f"{name}: a GPU tensor is needed")
    types = dtype if isinstance(dtype, tuple) else (dtype,)
    require(t.dtype in types, f"{name}: {t.dtype} given, {' or '.join(map(str, types))} needed")
    require(shape is None or tuple(t.shape) == tuple(shape),
            f"{name}: shape {tuple(t.shape)} given, {tuple(shape or ())} needed")
    require(device is None or t.device == device, f"{name}: on {t.device}, not on {device}")
    require(t.is_contiguous(), f"{name}: a contiguous tensor is needed")
    return t


class StreamSpace:
    """Workspace and zeroed counters, one of each per stream: calls on one stream
    are ordered, so they share; calls on different streams never do (those of a
    stream that is gone stay for the next one of its handle).  A call
    that is being captured into a graph gets its own, which the graph keeps
    (its counters are cleared within the graph, by a fill kernel)."""

    def __init__(self, device, workspace: int, counters: int):
        self.device, self.sizes = device, (max(16, workspace), max(16, counters))
        self._by_stream = {}

    def _make(self):
        w, c = self.sizes
        return (torch.empty(w, dtype=torch.uint8, device=self.device),
                torch.zeros((c + 3) // 4, dtype=torch.int32, device=self.device))

    def get(self, stream: int):
        """(workspace address, counters address, what keeps them alive)"""
        if torch.cuda.is_current_stream_capturing():
            pair = self._make()
            return pair[0].data_ptr(), pair[1].data_ptr(), pair
        got = self._by_stream.get(stream)
        if got is None:
            pair = self._make()
            got = self._by_stream[stream] = (pair[0].data_ptr(), pair[1].data_ptr(), pair)
        return got
