"""csrc/kv_index.h (the int8 paged cache's index arithmetic) compiled for the host, for tests."""

import ctypes
import functools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a8_codebook_quantized_rotate_b200", "csrc")

SRC = r"""
#include "kv_index.h"
using namespace w4a8;
extern "C" {
int first_key(int lo, int hi, int shift) { return kv_first_key(KvRange{lo, hi}, shift); }
}
"""


@functools.cache
def library():
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    out = os.path.join(ROOT, "_build", "kv_index_more")
    os.makedirs(out, exist_ok=True)
    src, so = os.path.join(out, "a.cc"), os.path.join(out, f"a{os.getpid()}.so")
    with open(src, "w") as f:
        f.write(SRC)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    os.remove(so)
    return lib
