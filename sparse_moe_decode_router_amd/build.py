"""Compile the HIP libraries for gfx950: the decode step (``libmoe_decode.so``)
and the serving operators around it (``libmoe_serve.so``).

Each is one translation unit (``csrc/moe_decode.hip``, ``csrc_serve/serve.hip``)
with the kernels and the C ABI declared in ``include/moe_decode.h`` and
``include/moe_serve.h``.  Packed-f32 instruction selection is
switched off for the device code.
"""
import hashlib
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "moe_decode.hip")
LIB = os.path.join(HERE, "libmoe_decode.so")
SERVE_SRC = os.path.join(HERE, "csrc_serve", "serve.hip")
SERVE_LIB = os.path.join(HERE, "libmoe_serve.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def command(out: str, extra=(), src: str = SRC) -> list:
    return [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
            "-Wall", "-Wno-unused-function",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
            "-I", os.path.join(HERE, "csrc_serve"), *extra, src, "-o", out]


def _build(src: str, lib: str, verbose: bool, extra) -> str:
    tmp = lib + ".tmp"
    cmd = command(tmp, extra, src)
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


def build(verbose: bool = False, extra=()) -> str:
    return _build(SRC, LIB, verbose, extra)


def build_serve(verbose: bool = False, extra=()) -> str:
    return _build(SERVE_SRC, SERVE_LIB, verbose, extra)


def source_digest() -> str:
    """Digest of the device sources: ties a stored hardware-counter reading
    to the kernels it was taken on."""
    h = hashlib.sha256()
    csrc = os.path.join(HERE, "csrc")
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name), "rb") as f:
            h.update(name.encode())
            h.update(f.read())
    return h.hexdigest()[:16]


if __name__ == "__main__":
    print(build(verbose=True, extra=sys.argv[1:]))
    print(build_serve(verbose=True, extra=sys.argv[1:]))
