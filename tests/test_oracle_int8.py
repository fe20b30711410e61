"""The oracle of the 8-bit integer path, pinned by brute force on tiny inputs."""

import math

import numpy as np
import pytest

from oracle import int8_ref as R
from oracle import w4a8_ref as O


def test_rows_agree_with_the_activation_oracle():
    x = np.random.default_rng(0).normal(size=(5, 512)).astype(np.float32)
    codes, s = R.quantize_rows(x, rotate=True)
    ref_codes, ref_s = O.quantize_activations(x)[:2]
    assert np.array_equal(codes, ref_codes) and np.array_equal(s, ref_s)


def test_rows_brute_force():
    x = np.array([[0.0] * 16, [1.0, -2.0, 0.5] + [0.0] * 13, [127.0, 0.5, 1.5, 2.5, -0.5] + [0.0] * 11], np.float32)
    codes, s = R.quantize_rows(x, rotate=False)
    assert s.tolist() == [0.0, np.float32(2.0) / np.float32(127.0), 1.0]
    assert not codes[0].any()
    assert codes[1, :3].tolist() == [round(1.0 / float(s[1])), -127, round(0.5 / float(s[1]))]
    assert codes[2, :5].tolist() == [127, 0, 2, 2, 0]   # ties to even


def test_product_triple_loop():
    rng = np.random.default_rng(1)
    x, w = rng.integers(-127, 128, (3, 16), dtype=np.int8), rng.integers(-127, 128, (4, 16), dtype=np.int8)
    sx, sw = rng.random(3, np.float32), rng.random(4, np.float32)
    y = R.product(x, sx, w, sw)
    for m in range(3):
        for n in range(4):
            acc = sum(int(x[m, k]) * int(w[n, k]) for k in range(16))
            assert y[m, n] == acc * float(sx[m]) * float(sw[n])


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_is_a_complex_turn(interleaved):
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=(2, 3, 64)), rng.random(64) + 0.5
    inv = 10000.0 ** (-np.arange(16) / 16)
    pos = np.array([0, 12345])
    y = R.norm_rope(x, w, 1e-6, pos, inv, interleaved, factor=1.25)
    for t in range(2):
        for h in range(3):
            rms = math.sqrt(sum(v * v for v in x[t, h]) / 64 + 1e-6)
            n = [v / rms * u for v, u in zip(x[t, h], w)]
            for i in range(16):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 16)
                z = complex(n[a], n[b]) * complex(math.cos(pos[t] * inv[i]), math.sin(pos[t] * inv[i])) * 1.25
                assert y[t, h, a] == pytest.approx(z.real, abs=1e-9) and y[t, h, b] == pytest.approx(z.imag, abs=1e-9)
            assert np.allclose(y[t, h, 32:], n[32:], atol=1e-12)


def _cache(rng, pages, heads, page, d):
    c = lambda: rng.integers(-127, 128, (pages, heads, page, d), dtype=np.int8)
    s = lambda: (rng.random((pages, heads)) + 0.1).astype(np.float32)
    return R.Cache(c(), c(), s(), s())


def test_update_token_by_token_meets_the_values():
    """A page written in two calls: the values of both are within half a step of the final scale plus the half
    step of the scale they were first written with; a page's first token drops the old scale."""
    rng = np.random.default_rng(3)
    c = _cache(rng, 3, 1, 16, 64)
    c.scales[0][:], c.scales[1][:] = 1e6, 1e6                 # stale: must not survive
    x = rng.normal(size=(20, 1, 64)).astype(np.float32)
    x[9] *= 5                                                 # grows the page's scale
    table, start = np.array([[2, 0]]), np.array([0, 8])
    R.update(c, x[:8], x[:8], table, start, np.array([8]))
    first = float(c.scales[0][2, 0])
    assert first == np.float32(np.abs(x[:8]).max()) / np.float32(127)
    R.update(c, x[8:], x[8:], table, np.array([0, 12]), np.array([20]))
    now = float(c.scales[0][2, 0])
    assert now == np.float32(np.abs(x[:16]).max()) / np.float32(127) and now > first
    v = c.values(0, 2, 0)
    assert np.abs(v[:8] - x[:8, 0]).max() <= 0.5 * first + 0.5 * now + 1e-6
    assert np.abs(v[8:] - x[8:16, 0]).max() <= 0.5 * now + 1e-6
    assert np.abs(c.values(1, 0, 0)[:4] - x[16:, 0]).max() <= 0.5 * float(c.scales[1][0, 0]) + 1e-6


def test_attention_brute_force():
    rng = np.random.default_rng(4)
    c = _cache(rng, 4, 2, 16, 64)
    q = rng.normal(size=(3, 4, 64))
    table, start, kv = np.array([[3, 1], [0, 2]]), np.array([0, 1, 3]), np.array([18, 5])
    out, absv, top, share = R.attention(q, c, table, start, kv, 0.01, window=4)
    for b, row, pos in ((0, 0, 17), (1, 1, 3), (1, 2, 4)):
        for h in range(4):
            num, den = np.zeros(64), 0.0
            for t in range(max(0, pos - 3), pos + 1):
                page, slot = table[b][t // 16], t % 16
                k = c.codes[0][page, h // 2, slot].astype(float) * float(c.scales[0][page, h // 2])
                v = c.codes[1][page, h // 2, slot].astype(float) * float(c.scales[1][page, h // 2])
                e = math.exp(0.01 * float(sum(a * d for a, d in zip(q[row, h], k))))
                num, den = num + e * v, den + e
            assert np.allclose(out[row, h], num / den, rtol=1e-9)
            assert (absv[row, h] >= np.abs(out[row, h]) - 1e-12).all()
