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
// Units that the tensor-memory attention kernel takes of a batch (0: the streaming kernel takes all of it).
int tensor_units(const int* q_len, const int* kv_len, int batch, int tokens, int group, int kv_heads, long long capacity,
                 int window, int d, int sms) {
  if (!kv_tiles_may_pay(tokens, batch, group, kv_heads, capacity, window, d, sms)) return 0;
  long long units = 0, work = 0, most = 0;
  for (int i = 0; i < batch; ++i) {
    const KvSeq s{0, q_len[i], kv_len[i], false};
    if (!kv_has_tiles(s, group)) continue;
    const KvTiles t = kv_tiles_of(s, group, window, kp_rows(d));
    units += t.tiles, work += t.row_keys, most = t.keys > most ? t.keys : most;
  }
  return kv_tiles_pay(units * kv_heads, work * kv_heads, most, d, sms) ? int(units * kv_heads) : 0;
}
long long tiles_bound(long long rows, long long batch, int tile_rows) { return kp_tiles_bound(rows, batch, tile_rows); }
long long first_item(long long c, long long total, long long ctas) { return ka_first_item(c, total, ctas); }
int item_cta(long long i, long long total, long long ctas) { return ka_item_cta(i, total, ctas); }
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
    for name in ("first_item", "tiles_bound"):
        getattr(lib, name).restype = ctypes.c_longlong
    lib.first_item.argtypes = lib.item_cta.argtypes = [ctypes.c_longlong] * 3
    lib.tiles_bound.argtypes = [ctypes.c_longlong] * 2 + [ctypes.c_int]
    lib.tensor_units.argtypes = [ctypes.c_void_p] * 2 + [ctypes.c_int] * 4 + [ctypes.c_longlong] + [ctypes.c_int] * 3
    return lib


def tensor_units(lens, q_heads, kv_heads, page, d, window=0, behind=0, sms=148):
    """Units that the tensor-memory attention kernel takes of sequences of (new tokens, tokens), under a block table of
    one page more than the longest needs; 0: the streaming kernel takes all."""
    q, kv = ((ctypes.c_int * len(lens))(*a) for a in zip(*lens))
    width = max(-(-n // page) for n in kv) + 1
    return library().tensor_units(q, kv, len(lens), sum(q) + behind, q_heads // kv_heads, kv_heads, width * page, window,
                                  d, min(sms, 160))
