"""Oracle of the 8-bit integer path (include/w4a8_int8.h): numpy, fp64, loops.

Integer decisions (scales, codes) are taken in fp32 like the kernels take
them, from values computed in fp64 and rounded once; everything that is a
real number is fp64.  Shares no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


# ---------------------------------------------------------------- int8 layer

def rotate_rows(x: np.ndarray) -> np.ndarray:
    """Each 256-block times H_256 / 16 (Sylvester order)."""
    h = np.ones((1, 1))
    for _ in range(8):
        h = np.block([[h, h], [h, -h]])
    r, k = x.shape
    return (np.asarray(x, np.float64).reshape(r, k // 256, 256) @ h).reshape(r, k) / 16.0


def codes_of(v: np.ndarray, s) -> np.ndarray:
    """clamp(round_half_even(fp32(v / s)), -127, 127) of fp32 values; 0 where s is 0."""
    v, s = np.asarray(v, F32), np.asarray(s, F32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.rint((v / s).astype(F32)), F32(0))
    return np.clip(q, -127, 127).astype(np.int8)


def quantize_rows(x: np.ndarray, rotate: bool):
    """(codes int8 [R, K], s fp32 [R])."""
    v = rotate_rows(x) if rotate else np.asarray(x, np.float64)
    v = v.astype(F32)
    s = (np.abs(v).max(axis=1) / F32(127)).astype(F32)
    return codes_of(v, s[:, None]), s


def product(x_q, s_x, w_q, s_w) -> np.ndarray:
    acc = x_q.astype(np.int64) @ w_q.astype(np.int64).T
    return acc.astype(np.float64) * s_x.astype(np.float64)[:, None] * s_w.astype(np.float64)[None, :]


# ---------------------------------------------------------------- heads

def norm_rope(x, weight, eps, positions, inv_freq, interleaved, factor=1.0):
    """x [T, H, D] -> fp64; weight None: no norm; inv_freq None: no rotation."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if inv_freq is None:
        return x
    half = len(inv_freq)
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(positions, np.float64)[:, None] * float(inv_freq[i])
        c, s = np.cos(angle) * factor, np.sin(angle) * factor
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# ---------------------------------------------------------------- cache

class Cache:
    """Codes [pages, heads, page, D] int8 and scales [pages, heads] fp32 of K and V."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.codes = [np.array(k_codes), np.array(v_codes)]
        self.scales = [np.array(k_scales, F32), np.array(v_scales, F32)]

    def write(self, kind: int, page_id: int, head: int, first: int, rows: np.ndarray) -> None:
        """New rows [n, D] (fp32 values) at places first .. first + n of a page."""
        rows = np.asarray(rows, F32)
        need = F32(np.abs(rows).max() / F32(127))
        old = F32(0) if first == 0 else self.scales[kind][page_id, head]
        new = max(old, need)
        codes = self.codes[kind][page_id, head]
        if first > 0 and new > old:
            ratio = F32(old / new)
            codes[:first] = np.rint((codes[:first].astype(F32) * ratio).astype(F32)).astype(np.int8)
        codes[first:first + len(rows)] = codes_of(rows, new)
        self.scales[kind][page_id, head] = new

    def values(self, kind: int, page_id: int, head: int) -> np.ndarray:
        return self.codes[kind][page_id, head].astype(np.float64) * float(self.scales[kind][page_id, head])


def update(cache: Cache, k, v, table, q_start, kv_len) -> None:
    """k (already normed and rotated), v [T, heads, D] into the cache."""
    heads, page = cache.codes[0].shape[1], cache.codes[0].shape[2]
    for b in range(len(kv_len)):
        n = int(q_start[b + 1] - q_start[b])
        pos0 = int(kv_len[b]) - n
        for p in range(pos0 // page, -(-int(kv_len[b]) // page) if n else 0):
            lo, hi = max(pos0, p * page), min(int(kv_len[b]), (p + 1) * page)
            if lo >= hi:
                continue
            rows = slice(int(q_start[b]) + lo - pos0, int(q_start[b]) + hi - pos0)
            for h in range(heads):
                for kind, x in ((0, k), (1, v)):
                    cache.write(kind, int(table[b][p]), h, lo - p * page, x[rows, h])


def attention(q, cache: Cache, table, q_start, kv_len, scale, window=0):
    """(out, absv, top, share): out [T, Hq, D] (NaN in rows of no sequence); absv, the same
    mean taken over |V|; per row, top, the largest sum_d |q_d K_d| * scale, and share, the
    number of keys times the largest weight * V scale."""
    q = np.asarray(q, np.float64)
    out = np.full(q.shape, np.nan)
    absv, top, share = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    heads, page = cache.codes[0].shape[1], cache.codes[0].shape[2]
    group = q.shape[1] // heads
    for b in range(len(kv_len)):
        n, length = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        for h in range(heads if n else 0):
            pages = [int(i) for i in table[b][: -(-length // page)]]
            k, v = (np.concatenate([cache.values(kind, i, h) for i in pages])[:length] for kind in (0, 1))
            vs = np.repeat([float(cache.scales[1][i, h]) for i in pages], page)[:length]
            for j in range(n):
                pos = length - n + j
                lo = max(0, pos - window + 1) if window else 0
                for g in range(group):
                    row, hd = int(q_start[b]) + j, h * group + g
                    s = k[lo:pos + 1] @ q[row, hd] * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[row, hd] = w @ v[lo:pos + 1]
                    absv[row, hd] = w @ np.abs(v[lo:pos + 1])
                    top[row, hd] = (np.abs(k[lo:pos + 1]) @ np.abs(q[row, hd])).max() * abs(scale)
                    share[row, hd] = (pos + 1 - lo) * (w * vs[lo:pos + 1]).max()
    return out, absv, top, share
