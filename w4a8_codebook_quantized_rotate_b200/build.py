"""Builds ``lib/libw4a8.so`` from ``csrc/`` with nvcc for sm_100a, and ``lib/w4a8_marshal.so``, the compiled part of
the binding, against it (in-tree)."""

from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "w4a8_api.cu")
OUT = os.path.join(PKG, "lib", "libw4a8.so")
MARSHAL_SRC = os.path.join(PKG, "csrc", "marshal.cpp")
MARSHAL_OUT = os.path.join(PKG, "lib", "w4a8_marshal.so")
MARSHAL_AGAINST = MARSHAL_OUT + ".against"

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    d = os.path.join(PKG, "csrc")
    return [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh", ".h"))] + [
        os.path.join(ROOT, "include", f) for f in ("w4a8.h", "w4a8_int8.h")]


def _fresh(out: str, srcs: list[str]) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(s) <= os.path.getmtime(out) for s in srcs)


def marshal_against() -> str:
    """What the binding's compiled part is compiled against, as text: this Python and this torch (whose C++ classes it
    uses, so another build of torch needs another one)."""
    import sys

    import torch
    return f"python {sys.version}\ntorch {torch.__version__} {torch.version.git_version} {os.path.dirname(torch.__file__)}\n"


def build_marshal(force: bool = False) -> str:
    """Compile the binding's compiled part (host C++ over the C ABI and torch's tensors) if it is not up to date: older
    than its sources, or compiled against another Python or torch than this one (kept beside it, in MARSHAL_AGAINST)."""
    headers = [os.path.join(ROOT, "include", f) for f in ("w4a8.h", "w4a8_int8.h")]
    against, was = marshal_against(), ""
    if os.path.exists(MARSHAL_AGAINST):
        with open(MARSHAL_AGAINST) as f:
            was = f.read()
    if not force and was == against and _fresh(MARSHAL_OUT, [MARSHAL_SRC, *headers]):
        return MARSHAL_OUT
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
           *(x for i in include for x in ("-isystem", i)), MARSHAL_SRC, "-o", MARSHAL_OUT + ".tmp",
           "-L", os.path.dirname(OUT), "-lw4a8", "-Wl,-rpath,$ORIGIN",
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib]
    subprocess.run(cmd, check=True)
    os.replace(MARSHAL_OUT + ".tmp", MARSHAL_OUT)
    with open(MARSHAL_AGAINST, "w") as f:
        f.write(against)
    return MARSHAL_OUT


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library, and the binding's compiled part, if any source is newer; return the library's path."""
    if not force and _fresh(OUT, sources()):
        build_marshal()
        return OUT
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", OUT + ".tmp", SRC]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(OUT + ".tmp", OUT)
    build_marshal(force)
    return OUT
