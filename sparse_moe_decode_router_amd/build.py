"""Compile the HIP libraries for gfx950: the decode step (``libmoe_decode.so``)
and the serving operators around it (``libmoe_serve.so``).

The first is one translation unit (``csrc/moe_decode.hip``), the second several
(``csrc_serve/*.hip``), compiled side by side; the C ABIs are declared in
``include/moe_decode.h`` and ``include/moe_serve.h``.  Packed-f32 instruction
selection is switched off for the device code.
"""
import hashlib
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "moe_decode.hip")
LIB = os.path.join(HERE, "libmoe_decode.so")
SERVE_SRCS = [os.path.join(HERE, "csrc_serve", name) for name in
              ("serve.hip", "shared.hip", "generate.hip")]
SERVE_LIB = os.path.join(HERE, "libmoe_serve.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def command(out: str, extra=(), src: str = SRC, kind: str = "-shared") -> list:
    return [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", kind,
            "-Wall", "-Wno-unused-function",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
            "-I", os.path.join(HERE, "csrc_serve"), *extra, src, "-o", out]


def _run(cmds, verbose: bool) -> None:
    """Runs commands side by side; all of them have to succeed."""
    for cmd in cmds if verbose else ():
        print(" ".join(cmd), flush=True)
    running = [subprocess.Popen(cmd) for cmd in cmds]
    for proc, code in [(p, p.wait()) for p in running]:
        if code:
            raise subprocess.CalledProcessError(code, proc.args)


def build(verbose: bool = False, extra=()) -> str:
    tmp = LIB + ".tmp"
    _run([command(tmp, extra)], verbose)
    os.replace(tmp, LIB)
    return LIB


def build_serve(verbose: bool = False, extra=()) -> str:
    objects = [src[:-len(".hip")] + ".o" for src in SERVE_SRCS]
    tmp = SERVE_LIB + ".tmp"
    _run([command(o, extra, src, "-c") for o, src in zip(objects, SERVE_SRCS)], verbose)
    _run([[HIPCC, "--offload-arch=gfx950", "-shared", *objects, "-o", tmp]], verbose)
    for o in objects:
        os.remove(o)
    os.replace(tmp, SERVE_LIB)
    return SERVE_LIB


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
