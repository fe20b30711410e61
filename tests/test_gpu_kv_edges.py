"""Edges of the int8 paged cache's calls (include/w4a8_int8.h), against the
oracle and the bars of test_gpu_kv.py, or against the same call without the
edge, bit for bit."""

import numpy as np
import pytest
import torch

from oracle import int8_ref as R
from test_gpu_kv import INV, Batch, bf16, check_attention, dev

pytestmark = pytest.mark.gpu

# (lens, query heads, key heads, least) of a batch for the streaming kernel, and one whose rows and keys pay for the
# tensor-memory kernel at every head size
FEW, MANY = ([(1, 400), (8, 90)], 4, 2, 2.0 ** -39), ([(200, 1300)], 32, 16, 2.0 ** -32)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hq,hk,least,powers", [(*FEW, (-124, -112, 112, 118, 124)), (*MANY, (-124, 124))])
def test_queries_at_the_ends_of_the_range(lib, d, lens, hq, hk, least, powers):
    """Queries of 2^-124 to 2^124 (finite, up to 2^126) and K scales that bring the scores back to a few units: the
    row's power of two must reach them all."""
    b = Batch(lens, hk, 16, d, 80 + d)
    x, _ = bf16(b.rng, b.t, hq, d)
    k_scales = b.ref.scales[0].copy()
    for power in powers:
        q = (x.float() * 2.0 ** power).to(torch.bfloat16)
        assert q.isfinite().all()
        b.ref.scales[0] = (k_scales.astype(np.float64) * 2.0 ** -power).astype(np.float32)
        got = lib.kv_attention(q, b.cache(lib), *b.args())
        assert lib.get_device_error() == 0
        check_attention(got, *R.attention(q.double().cpu().numpy(), b.ref, b.table, b.start, b.kv_len, d ** -0.5), least=least)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hq,hk,least", [FEW, MANY])
@pytest.mark.parametrize("power,window", [(118, 0), (34, 70), (30, 0)])
def test_one_key_takes_all_the_weight(lib, d, lens, hq, hk, least, power, window):
    """Scores of about 2^22, 2^26 and 2^110: a row's largest score is far ahead, and its output that key's value, where
    the two largest are further apart than twice what fp32 loses (2^-18 of sum |q_d K_d| scale each, so 2^-16 of it and 64
    more leave the others below 2^-90).  The value: p vs rounded to fp16 (2^-11), the sum (2^-16), the output (2^-8)."""
    b = Batch(lens, hk, 16, d, 90 + d)
    x, _ = bf16(b.rng, b.t, hq, d)
    q = (x.float() * 2.0 ** power).to(torch.bfloat16)
    b.ref.scales[0] *= np.float32(2.0 ** -8)
    got = lib.kv_attention(q, b.cache(lib), *b.args(), window=window).double().cpu().numpy()
    assert lib.get_device_error() == 0 and np.isfinite(got).all()
    q, group, seen = q.double().cpu().numpy(), hq // hk, 0
    for i, n in enumerate(b.q_len):
        length = int(b.kv_len[i])
        pages = b.table[i][:-(-length // 16)]
        for h in range(hk):
            k, v = (np.concatenate([b.ref.values(kind, p, h) for p in pages])[:length] for kind in (0, 1))
            for j in range(n):
                end = length - n + j + 1
                keys = slice(max(0, end - window) if window else 0, end)
                rows = q[b.start[i] + j, h * group:(h + 1) * group]
                s, top = rows @ k[keys].T * d ** -0.5, (np.abs(rows) @ np.abs(k[keys]).T).max(1) * d ** -0.5
                best = np.partition(s, -2, axis=1)
                for g in np.flatnonzero(best[:, -1] - best[:, -2] > 2.0 ** -16 * top + 64):
                    want = v[keys][np.argmax(s[g])]
                    out = got[b.start[i] + j, h * group + g]
                    assert (np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * np.abs(want) + 2.0 ** -73).all()
                    seen += 1
    assert seen > 0.9 * b.t * hq


@pytest.mark.parametrize("good,bad", [(32, (0, 10 ** 6)), (32, (0, -3)), (32, (5, 40)), (64, (0, 10 ** 6)), (700, (0, 10 ** 6))])
def test_a_bad_sequence_behind_many_is_reported(lib, good, bad):
    """The last sequence's numbers do not fit, behind 32 or more that fill every unit of the update's launch: its end
    past the rows, or a length that the table has no places for.  The others' results are those without it."""
    b = Batch([(1, 1 + i % 20) for i in range(good)], 2, 16, 64, 100)
    k, _ = bf16(b.rng, b.t, 2, 64)
    q, _ = bf16(b.rng, b.t, 4, 64)
    one, two = b.cache(lib), b.cache(lib)
    want = lib.kv_update(one, k, k, *b.args(), q=q)
    assert lib.get_device_error() == 0
    table = dev(np.concatenate([b.table, b.table[:1]]))
    start = dev(np.append(b.start, b.start[-1] + bad[0]).astype(np.int32))
    kv = dev(np.append(b.kv_len, bad[1]).astype(np.int32))
    got = lib.kv_update(two, k, k, table, start, kv, q=q)
    assert lib.get_device_error() == 8                        # W4A8_ERR_INPUT
    assert torch.equal(got, want)
    assert torch.equal(one.k_codes, two.k_codes) and torch.equal(one.k_scales, two.k_scales)
    out = lib.kv_attention(want, one, *b.args())
    assert lib.get_device_error() == 0
    assert torch.equal(lib.kv_attention(want, one, table, start, kv), out) and lib.get_device_error() == 8


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,hq,hk,window", [
    ([(1, 300 + 13 * i) for i in range(12)] + [(5, 411), (3, 20), (1, 7)], 4, 2, 37),      # a few rows
    ([(1, 290), (1, 291), (1, 305), (2, 1000)], 4, 2, 1),
    ([(900, 1700), (1, 333)], 32, 16, 100),                                                # many: the other kernel
])
def test_pages_behind_the_window_may_be_gone(lib, d, page, lens, hq, hk, window):
    """Entries of pages that every new token's window has passed are not read: -1 there is no error, and what the pages
    held is not looked at."""
    b = Batch(lens, hk, page, d, page + d + window)
    q, _ = bf16(b.rng, b.t, hq, d)
    want = lib.kv_attention(q, b.cache(lib), *b.args(), window=window)
    assert lib.get_device_error() == 0
    gone = []
    for i, n in enumerate(b.q_len):
        first = max(0, int(b.kv_len[i]) - n - window + 1)     # the first key that a token of the sequence sees
        gone += b.table[i, :first // page].tolist()
        b.table[i, :first // page] = -1
    assert len(gone) > 0
    cache = b.cache(lib)
    for t in (cache.k_scales, cache.v_scales):
        t[gone] = float("nan")
    for bad in (-1, b.pages, 2 ** 31 - 1):
        b.table[b.table == -1] = bad
        assert torch.equal(lib.kv_attention(q, cache, *b.args(), window=window), want)
        assert lib.get_device_error() == 0
        b.table[b.table == bad] = -1


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hq,hk", [FEW[:3], MANY[:3], ([(1, 3000)], 8, 2), ([(200, 1300), (1, 500), (3, 40)], 32, 16)])
def test_attention_in_place(lib, d, lens, hq, hk):
    """The output over its queries, parts of a longer row: the bits of a call with an output of its own."""
    b = Batch(lens, hk, 16, d, 110 + d, behind=2)
    rows, _ = bf16(b.rng, b.t, hq + 3, d)
    q, cache = rows[:, 1:1 + hq], b.cache(lib)
    want, rest = lib.kv_attention(q, cache, *b.args()), rows.clone()
    n = int(b.start[-1])
    lib.kv_attention(q, cache, *b.args(), out=q)
    assert lib.get_device_error() == 0
    rest[:n, 1:1 + hq] = want[:n]
    assert torch.equal(rows, rest)
    with pytest.raises(lib.W4A8Error):
        lib.kv_attention(q, cache, *b.args(), out=q.as_strided(q.shape, (hq * d, d, 1)))


def test_strides_of_one_token_or_one_head_do_not_matter(lib):
    """In place, where a dimension of one has another stride than the input's."""
    w, inv = dev(np.ones(128, np.float32)), dev(INV[64])
    for t, h, strides in ((1, 4, (4096, 128, 1)), (3, 1, (512, 4096, 1))):
        x, _ = bf16(np.random.default_rng(111), t, 4, 128)
        x = x[:, :h]
        pos = torch.arange(t, dtype=torch.int32, device="cuda")
        want, _ = lib.qk_norm_rope(x, None, pos, w, inv_freq=inv)
        lib.qk_norm_rope(x, None, pos, w, inv_freq=inv, q_out=x.as_strided(x.shape, strides))
        assert torch.equal(x, want) and lib.get_device_error() == 0
