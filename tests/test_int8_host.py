"""Host-side checks of the 8-bit integer path that need no GPU: the entry
points of include/w4a8_int8.h are exported, sizes follow from the layout, bad
arguments are refused before any launch, and the kernels' index arithmetic
(csrc/kv_index.h, compiled here for the host) keeps every access in range."""

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w4a8_int8.h")
CSRC = os.path.join(ROOT, "w4a8_codebook_quantized_rotate_b200", "csrc")
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
P = 4096            # an aligned address that nothing reads


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("factor", ctypes.c_float)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class BatchDesc(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("batch", ctypes.c_int64), ("tokens", ctypes.c_int64)]


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from w4a8_codebook_quantized_rotate_b200 import binding
    binding.load_library()
    return binding


@pytest.fixture(scope="module")
def lib(B):
    return B.load_library()


def test_exports(B, lib):
    names = re.findall(r"^\s*(?:size_t|w4a8_status)\s+(w4a8_\w+)\s*\(", open(HEADER).read(), re.M)
    assert len(names) == 9
    for name in names:
        assert hasattr(lib, name) and name in B.EXPORTS


def test_header_is_plain_c(B):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = '#include "w4a8_int8.h"\nint main(void) { return w4a8_int8_linear_workspace_bytes(1, 7, 1) == 0 ? 0 : 1; }\n'
    out = os.path.join(ROOT, "_build", "abi_int8")
    os.makedirs(out, exist_ok=True)
    with open(os.path.join(out, "a.c"), "w") as f:
        f.write(src)
    libdir = os.path.dirname(B.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.dirname(HEADER),
                    os.path.join(out, "a.c"), "-o", os.path.join(out, "a"), "-L", libdir, "-lw4a8",
                    "-Wl,-rpath," + libdir], check=True)
    assert subprocess.run([os.path.join(out, "a")]).returncode == 0



def test_int8_layer_refusals(lib):
    ws = lib.w4a8_int8_linear_workspace_bytes(5, 512, 64)
    assert ws >= 5 * 512 + 5 * 4
    for m, k, n in ((0, 512, 64), (5, 500, 64), (5, 0, 64), (5, 512, 0), (5, 32784, 64), (5, 512, 2 ** 24 + 1),
                    (65535 * 256 + 1, 512, 64)):
        assert lib.w4a8_int8_linear_workspace_bytes(m, k, n) == 0
        assert lib.w4a8_int8_gemm(P, P, m, P, P, n, k, P, None) == SHAPE
        assert lib.w4a8_int8_linear(P, m, k, 0, P, P, n, P, P, 1 << 40, None) == SHAPE
    assert lib.w4a8_int8_linear(P, 5, 272, 1, P, P, 64, P, P, 1 << 30, None) == SHAPE   # rotation needs K % 256
    assert lib.w4a8_int8_linear_workspace_bytes(5, 272, 64) > 0
    assert lib.w4a8_int8_linear(P, 5, 512, 1, P, P, 64, P, P, ws - 1, None) == WORKSPACE
    for i in (0, 1, 3, 4, 7):
        a = [P, P, 5, P, P, 64, 512, P, None]
        a[i] = None
        assert lib.w4a8_int8_gemm(*a) == NULL
        a[i] = P + 8
        assert lib.w4a8_int8_gemm(*a) == ALIGN
    for i in (0, 4, 5, 7, 8):
        a = [P, 5, 512, 1, P, P, 64, P, P, 1 << 30, None]
        if i not in (1, 2, 3, 6):
            a[i] = None
            assert lib.w4a8_int8_linear(*a) == NULL
            a[i] = P + 8
            assert lib.w4a8_int8_linear(*a) == ALIGN
    assert lib.w4a8_int8_quantize(None, 0, 4, 512, 0, P, P, None) == NULL
    assert lib.w4a8_int8_quantize(P, 0, 4, 520, 0, P, P, None) == SHAPE
    assert lib.w4a8_int8_quantize(P, 0, 4, 528, 1, P, P, None) == SHAPE
    assert lib.w4a8_int8_quantize(P, 0, 0, 512, 0, P, P, None) == SHAPE
    assert lib.w4a8_int8_quantize(P, 0, 4, 512, 0, P + 4, P, None) == ALIGN


def _heads(B, heads=4, d=128, data=P, token=None, head=None):
    return Heads(data, heads * d if token is None else token, d if head is None else head, heads)


def _qk(B, lib, q=None, k=None, t=3, d=128, qw=P, kw=P, pos=P, rope=None, qo=None, ko=None):
    r = rope or Rope(P, 64, 0, 1.0)
    ref = lambda x, y: ctypes.byref(x if x is not None else y)
    return lib.w4a8_qk_norm_rope(ref(q, _heads(B)), ref(k, _heads(B, 2)), t, d, qw, kw, 1e-6, pos, ctypes.byref(r),
                                 ref(qo, _heads(B)), ref(ko, _heads(B, 2)), None)


def test_norm_rope_refusals(B, lib):
    none = Heads(None, 0, 0, 0)
    assert _qk(B, lib, q=none, k=none) == NULL
    assert _qk(B, lib, qo=none) == NULL
    assert _qk(B, lib, pos=None) == NULL
    assert _qk(B, lib, t=0) == SHAPE
    assert _qk(B, lib, d=96) == SHAPE
    assert _qk(B, lib, q=_heads(B, token=516)) == SHAPE          # strides are multiples of 8
    assert _qk(B, lib, q=_heads(B, head=64)) == SHAPE            # heads overlap
    assert _qk(B, lib, q=_heads(B, 3)) == SHAPE                  # q_out has 4 heads
    assert _qk(B, lib, q=_heads(B, data=P + 8)) == ALIGN
    assert _qk(B, lib, qw=P + 4) == ALIGN
    assert _qk(B, lib, pos=P + 2) == ALIGN
    for rot in (0, 8, 24, 144):
        assert _qk(B, lib, rope=Rope(P, rot, 0, 1.0)) == SHAPE
    assert _qk(B, lib, rope=Rope(P + 4, 64, 0, 1.0)) == ALIGN


def _cache(B, pages=10, heads=2, page=16, d=128, data=P):
    return CacheDesc(data, P, P, P, pages, heads, page, d)


def _batch(B, batch=2, tokens=3, width=4, table=P):
    return BatchDesc(table, width, P, P, batch, tokens)


def _update(B, lib, cache=None, batch=None, k=None, v=None, q=None, qo=None, rope=None, pos=None):
    none = Heads(None, 0, 0, 0)
    r = rope or Rope(P, 64, 0, 1.0)
    ref = ctypes.byref
    return lib.w4a8_kv_update(ref(cache or _cache(B)), ref(batch or _batch(B)), ref(k or _heads(B, 2)), ref(v or _heads(B, 2)),
                              ref(q or none), None, P, 1e-6, pos, ref(r), ref(qo or none), None)


def _attend(B, lib, cache=None, batch=None, q=None, out=None, window=0, ws=P, nbytes=1 << 40):
    ref = ctypes.byref
    return lib.w4a8_kv_attention(ref(q or _heads(B)), ref(cache or _cache(B)), ref(batch or _batch(B)), 0.1, window,
                                 ref(out or _heads(B)), ws, nbytes, None)


BAD_CACHES = [dict(pages=0), dict(pages=2 ** 31 // 32), dict(heads=0), dict(page=24), dict(page=8), dict(page=256),
              dict(d=96), dict(d=512)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_cache_refusals(B, lib, bad):
    c = _cache(B, **bad)
    assert _update(B, lib, cache=c) == SHAPE
    assert _attend(B, lib, cache=c) == SHAPE
    assert lib.w4a8_kv_dequant(ctypes.byref(c), P, 2, P, P, None) == SHAPE


def test_update_and_attention_refusals(B, lib):
    none = Heads(None, 0, 0, 0)
    assert _update(B, lib, cache=_cache(B, data=None)) == NULL
    assert _update(B, lib, cache=_cache(B, data=P + 8)) == ALIGN
    assert _update(B, lib, batch=_batch(B, table=None)) == NULL
    assert _update(B, lib, batch=_batch(B, table=P + 2)) == ALIGN
    for bad in (dict(batch=0), dict(batch=65537), dict(tokens=0), dict(tokens=2 ** 24 + 1), dict(width=0),
                dict(width=2 ** 27), dict(width=2 ** 26 + 1)):
        assert _update(B, lib, batch=_batch(B, **bad)) == SHAPE
        assert _attend(B, lib, batch=_batch(B, **bad)) == SHAPE
    shared = Heads(P, 0, 128, 4), Heads(P, 504, 128, 4), Heads(P, 128, 128, 4), Heads(P, 128, 256, 4)   # of 3 tokens
    for rows in shared:                                          # rows of an output that share memory
        assert _attend(B, lib, out=rows) == SHAPE
        assert _update(B, lib, q=_heads(B), qo=rows) == SHAPE
        assert lib.w4a8_qk_norm_rope(ctypes.byref(_heads(B)), None, 3, 128, None, None, 1e-6, None, None,
                                     ctypes.byref(rows), None, None) == SHAPE
    assert _update(B, lib, k=_heads(B, 4)) == SHAPE              # the cache has 2 heads
    assert _update(B, lib, q=_heads(B)) == NULL                  # q without q_out
    assert _update(B, lib, q=_heads(B), qo=_heads(B, 3)) == SHAPE
    assert _update(B, lib, rope=Rope(P, 40, 0, 1.0)) == SHAPE
    assert _update(B, lib, pos=P + 1) == ALIGN
    assert _attend(B, lib, q=none) == NULL
    assert _attend(B, lib, ws=None) == NULL
    assert _attend(B, lib, ws=P + 8) == ALIGN
    assert _attend(B, lib, window=-1) == SHAPE
    assert _attend(B, lib, q=_heads(B, 3), out=_heads(B, 3)) == SHAPE    # 3 heads over 2
    assert _attend(B, lib, out=_heads(B, 6)) == SHAPE
    need = lib.w4a8_kv_attention_workspace_bytes(3, 4, 2, 128)
    assert need > 0 and _attend(B, lib, nbytes=need - 1) == WORKSPACE
    assert lib.w4a8_kv_attention_workspace_bytes(3, 5, 2, 128) == 0
    assert lib.w4a8_kv_attention_workspace_bytes(3, 258, 2, 128) == 0    # 129 heads to a key head
    assert lib.w4a8_kv_attention_workspace_bytes(3, 4, 2, 80) == 0
    c = _cache(B)
    assert lib.w4a8_kv_dequant(ctypes.byref(c), None, 2, P, P, None) == NULL
    assert lib.w4a8_kv_dequant(ctypes.byref(c), P, 0, P, P, None) == SHAPE
    assert lib.w4a8_kv_dequant(ctypes.byref(c), P + 2, 2, P, P, None) == ALIGN


def test_binding_refuses_before_the_library(B):
    """What needs no GPU to be refused: tensors elsewhere or of another kind, and no tensors."""
    x, q = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, None)                               # not on a GPU
    with pytest.raises(ValueError):
        B.qk_norm_rope(None, [1, 2])
    with pytest.raises(ValueError):
        B.int8_gemm(x, None, x, None)
    with pytest.raises(ValueError):
        B.int8_linear(x[0], x, None)
    with pytest.raises(ValueError):
        B.KvCache.of(*(torch.zeros(2, 2, 16, 64, dtype=torch.int8),) * 2, *(torch.zeros(2, 2),) * 2)
    with pytest.raises(TypeError):
        B._m().int8_gemm(x, x)


def test_rope_frequencies(B):
    plain, f = B.rope_frequencies(64, base=500000.0, device="cpu")
    assert f == 1.0 and plain.dtype == torch.float64
    assert np.allclose(plain.numpy(), 500000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    lin, _ = B.rope_frequencies(64, base=500000.0, scaling="linear", factor=8.0, device="cpu")
    assert torch.equal(lin, plain / 8)
    ntk, _ = B.rope_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    base, _ = B.rope_frequencies(64, device="cpu")
    assert ntk[0] == 1.0 and float(ntk[-1] * 8 / base[-1]) == pytest.approx(1.0, rel=1e-12)
    yarn, f = B.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    assert f == pytest.approx(0.1 * np.log(4.0) + 1)
    r = (yarn / base).numpy()
    assert r[0] == 1.0 and r[-1] == pytest.approx(0.25) and (np.diff(r) <= 1e-12).all()
    turns = 4096 * base.numpy() / (2 * np.pi)
    assert (r[turns > 40] == 1.0).all() and np.allclose(r[turns < 0.7], 0.25)
    for bad in (dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            B.rope_frequencies(device="cpu", **bad)


# ---------------------------------------------------------------- csrc/kv_index.h

SRC = r"""
#include "kv_index.h"
using namespace w4a8;
extern "C" {
int pays(long long units, long long row_keys, long long most, int d, int sms) { return kv_tiles_pay(units, row_keys, most, d, sms); }
void seq(int start, int end, int kv, long long tokens, long long table, int* out) {
  KvSeq s = kv_seq(start, end, kv, tokens, table);
  out[0] = s.start; out[1] = s.q_len; out[2] = s.kv_len; out[3] = s.bad;
}
int touched(int q, int kv, int shift) { KvSeq s{0, q, kv, false}; return kv_touched(s, shift); }
int first(int q, int kv, int shift) { KvSeq s{0, q, kv, false}; return kv_first_page(s, shift); }
long long bound(long long tokens, long long batch, int page) { return kv_touched_bound(tokens, batch, page); }
void range(int q, int kv, int j0, int j1, int window, int* out) {
  KvSeq s{0, q, kv, false}; KvRange r = kv_range(s, j0, j1, window); out[0] = r.lo; out[1] = r.hi;
}
}
"""


@pytest.fixture(scope="module")
def index():
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    out = os.path.join(ROOT, "_build", "kv_index")
    os.makedirs(out, exist_ok=True)
    with open(os.path.join(out, "a.cc"), "w") as f:
        f.write(SRC)
    so = os.path.join(out, "a.so")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(out, "a.cc"), "-o", so], check=True)
    h = ctypes.CDLL(so)
    h.bound.restype = ctypes.c_longlong
    h.bound.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int]
    h.seq.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong] * 2 + [ctypes.c_void_p]
    return h


def test_sequences_that_do_not_fit_are_left_out(index):
    def seq(start, end, kv, tokens=100, table=640):
        out = (ctypes.c_int * 4)()
        index.seq(start, end, kv, tokens, table, out)
        return list(out)
    assert seq(3, 7, 50) == [3, 4, 50, 0]
    assert seq(7, 7, 0) == [7, 0, 0, 0]
    assert seq(90, 100, 640) == [90, 10, 640, 0]
    for bad in ((-1, 3, 50), (7, 3, 50), (95, 101, 50), (3, 7, 3), (3, 7, -1), (3, 7, 641),
                (0, 2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1, 5)):
        assert seq(*bad) == [0, 0, 0, 1], bad


def test_touched_pages(index):
    rng = np.random.default_rng(0)
    for _ in range(300):
        shift = int(rng.integers(4, 8))
        page = 1 << shift
        lens = []
        for _ in range(int(rng.integers(1, 6))):
            kv = int(rng.integers(1, 400))
            lens.append((int(rng.integers(0, kv + 1)), kv))
        total = 0
        for q, kv in lens:
            want = {t // page for t in range(kv - q, kv)}
            n = index.touched(q, kv, shift)
            assert n == len(want)
            if q:
                assert index.first(q, kv, shift) == min(want)
            total += n
        tokens = sum(q for q, _ in lens)
        assert total <= index.bound(tokens, len(lens), page) <= max(tokens, 1)


def test_key_ranges(index):
    out = (ctypes.c_int * 2)()
    for q, kv, window in ((1, 1, 0), (5, 9, 0), (5, 9, 3), (9, 9, 100), (4, 50, 1)):
        for j0 in range(q):
            for j1 in range(j0, q):
                index.range(q, kv, j0, j1, window, out)
                seen = [t for j in range(j0, j1 + 1) for t in range(kv - q + j + 1)
                        if not window or t > kv - q + j - window]
                assert [out[0], out[1]] == [min(seen), max(seen) + 1]


def test_every_item_has_one_cta():
    """The split of a kernel's items over CTAs: contiguous shares that cover
    every item once, none empty, and the CTA named for an item holds it."""
    first = lambda c, total, ctas: total * c // ctas
    of = lambda i, total, ctas: ((i + 1) * ctas + total - 1) // total - 1
    for total in (1, 2, 3, 7, 147, 148, 149, 1000, 4097):
        ctas = min(total, 148)
        edges = [first(c, total, ctas) for c in range(ctas + 1)]
        assert edges[0] == 0 and edges[-1] == total and all(a < b for a, b in zip(edges, edges[1:]))
        for i in range(total):
            c = of(i, total, ctas)
            assert edges[c] <= i < edges[c + 1]


def test_choice_of_the_attention_kernel(index):
    """Measured on both sides (us, streaming / tensor-memory): new tokens, heads, D, keys, units."""
    import ctypes
    f = index.pays
    f.argtypes, f.restype = [ctypes.c_longlong] * 3 + [ctypes.c_int] * 2, ctypes.c_int
    for q, hq, hk, d, keys, stream, tensor in ((130, 32, 8, 128, 230, 14, 28), (500, 8, 2, 128, 6000, 90, 58),
                                               (260, 12, 1, 256, 6000, 133, 70), (260, 24, 4, 256, 6000, 250, 72),
                                               (64, 24, 4, 64, 6000, 30, 46), (260, 8, 2, 64, 6000, 36, 47)):
        rows = q * hq // hk
        units = -(-rows // (256 if d <= 128 else 128)) * hk
        assert bool(f(units, rows * (keys + 512) * hk, keys, d, 148)) == (tensor < stream)
    assert not f(0, 0, 0, 128, 148)
    assert f(2 ** 23, 2 ** 60, 2 ** 30, 256, 148)            # nothing wraps at the largest sizes
