"""GPU parity of the attention block's steps (w4a8_qk_norm_rope, w4a8_kv_update,
w4a8_kv_dequant, w4a8_kv_attention) against oracle/int8_ref.py.

Bars:
  * norm and rotation: bf16 rounds by at most 2^-8 of the value; before it the
    fp32 sum of at most 256 squares (8 in a lane, 5 shuffles), the reciprocal
    root, two products, the angle (a fraction of a turn rounded to fp32,
    2 pi 2^-25) and the turn of a pair (a, b) stay within 2^-19 (|a| + |b|);
  * cache: scales and codes of V, and of K without norm and rotation, are
    bit-exact (fp32 decisions on the same inputs), recoded ones too; with
    them a scale is within 2^-19 and a code within one step, on at most 3e-3
    of the codes (a value off by 127 * 2^-19 of a step changes code with
    probability 5e-4);
  * attention: bf16 output 2^-8 |out|; p vs is rounded to fp16 (2^-11) and
    p, the sum and the accumulation are fp32 (2^-16 in all), each against the
    mean of |V| under the same weights; a score's fp32 error is within 2^-18
    of sum |q_d K_d| scale and moves the weights by twice that.  fp16 holds
    p vs with the row's largest at 2^14 or more (2^15 less one step of its
    running maximum), so a subnormal one is off by at most 2^-25, 2^-39 of the
    largest; times a code (2^7), for every key.  The tensor-memory kernel puts
    the largest at 2^7 (and keeps the reference until it grows by 2^8), which
    makes that 2^-32.  V scales below 2^-80 count as 0, and a key without a V
    scale enters the reference as one of 2^-80, so what is below 2^-80 2^7 is
    not kept: 2^-73 in absolute terms.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import int8_ref as R

pytestmark = pytest.mark.gpu

INV = {rot: 10000.0 ** (-np.arange(0, rot, 2) / rot) for rot in (16, 32, 64, 128, 256)}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(rng, *shape, scale=1.0):
    """(tensor, its fp64 values)"""
    bits = synth.f32_to_bf16_bits((rng.normal(size=shape) * scale).astype(np.float32))
    return dev(bits.view(np.int16)).view(torch.bfloat16), synth.bf16_bits_to_f32(bits).astype(np.float64)


def check_heads(got, ref, pair):
    got = got.double().cpu().numpy()
    over = np.abs(got - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -19 * pair
    assert over.max() <= 0, f"{(over > 0).sum()} values off, worst {over.max():.3e}"


def pair_size(x, w, rot, interleaved, factor):
    """|a| + |b| of each value's pair after the norm (|x| where none)."""
    n = np.abs(R.norm_rope(x, w, 1e-6, None, None, False)) * max(1.0, factor)
    if rot:
        y, h = n.copy(), rot // 2
        if interleaved:
            y[..., 0:rot:2] = y[..., 1:rot:2] = n[..., 0:rot:2] + n[..., 1:rot:2]
        else:
            y[..., :h] = y[..., h:rot] = n[..., :h] + n[..., h:rot]
        n = y
    return n


@pytest.mark.parametrize("t,hq,hk,d,rot,interleaved", [
    (1, 1, 1, 64, 16, False), (3, 8, 2, 64, 64, True), (5, 24, 4, 256, 64, False), (7, 32, 8, 128, 128, True),
    (9, 7, 1, 128, 32, False), (2, 3, 3, 256, 256, False), (4, 5, 5, 256, 256, True), (33, 40, 8, 128, 128, False),
    (6, 4, 2, 128, 0, False)])
def test_norm_rope(lib, t, hq, hk, d, rot, interleaved):
    rng = np.random.default_rng(t * d + rot)
    q, qx = bf16(rng, t, hq, d, scale=3.0)
    k, kx = bf16(rng, t, hk, d)
    qw, kw = (rng.random(d) + 0.5).astype(np.float32), (rng.random(d) + 0.5).astype(np.float32)
    pos = rng.integers(0, 10 ** 6, t).astype(np.int32)
    pos[0] = 0
    inv = INV[rot] if rot else None
    for wq, wk, factor in ((qw, kw, 1.0), (None, kw, 1.2)):
        qo, ko = lib.qk_norm_rope(q, k, dev(pos), q_weight=None if wq is None else dev(wq), k_weight=dev(wk),
                                  inv_freq=None if inv is None else dev(inv), interleaved=interleaved, rope_factor=factor)
        for got, x, w in ((qo, qx, wq), (ko, kx, wk)):
            check_heads(got, R.norm_rope(x, w, 1e-6, pos, inv, interleaved, factor), pair_size(x, w, rot, interleaved, factor))
    assert lib.get_device_error() == 0


def test_norm_rope_strided_in_place_and_alone(lib):
    """Parts of one projection's rows, in place; k alone; a row of zeros."""
    rng = np.random.default_rng(5)
    t, hq, hk, d = 6, 6, 2, 128
    rows, x = bf16(rng, t, (hq + 2 * hk) * d + 8)
    rows[2], x[2] = 0, 0
    part = lambda a, i, n: a[:, i * d:(i + n) * d].reshape(t, n, d)
    q, k = rows[:, :hq * d].unflatten(1, (hq, d)), rows[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    rest = rows[:, (hq + hk) * d:].clone()
    w, pos = np.ones(d, np.float32), np.arange(t, dtype=np.int32) * 1000
    alone = lib.qk_norm_rope(None, k, dev(pos), k_weight=dev(w), inv_freq=dev(INV[64]))
    lib.qk_norm_rope(q, k, dev(pos), q_weight=dev(w), k_weight=dev(w), inv_freq=dev(INV[64]), q_out=q, k_out=k)
    assert alone[0] is None and torch.equal(alone[1], k)
    for got, v in ((q, part(x, 0, hq)), (k, part(x, hq, hk))):
        check_heads(got, R.norm_rope(v, w, 1e-6, pos, INV[64], False), pair_size(v, w, 64, False, 1.0))
    assert torch.equal(rows[:, (hq + hk) * d:], rest)


# ---------------------------------------------------------------- cache

class Batch:
    """Random sequences and a cache that holds them (codes and scales of everything random)."""

    def __init__(self, lens, hk, page, d, seed, spare=3, scale=0.02, behind=0):
        rng = self.rng = np.random.default_rng(seed)
        self.q_len, self.kv_len = [a for a, _ in lens], np.array([b for _, b in lens], np.int32)
        self.start = np.concatenate([[0], np.cumsum(self.q_len)]).astype(np.int32)
        self.t = int(self.start[-1]) + behind
        n = [-(-int(v) // page) for v in self.kv_len]
        self.pages = sum(n) + spare
        order, at = rng.permutation(self.pages), 0
        self.table = np.full((len(lens), max(n) + 1), -1, np.int32)
        for i, c in enumerate(n):
            self.table[i, :c] = order[at:at + c]
            at += c
        shape = (self.pages, hk, page, d)
        code = lambda: np.clip(np.rint(rng.normal(size=shape) * 40), -127, 127).astype(np.int8)
        s = lambda: ((rng.random(shape[:2]) + 0.25) * scale).astype(np.float32)
        self.ref = R.Cache(code(), code(), s(), s())

    def cache(self, lib):
        r = self.ref
        return lib.KvCache.of(*(dev(a) for a in (r.codes[0], r.codes[1], r.scales[0], r.scales[1])))

    def args(self):
        return dev(self.table), dev(self.start), dev(self.kv_len)


RAGGED = [(1, 1), (1, 16), (1, 17), (5, 40), (33, 33), (0, 9), (64, 130), (2, 33)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_update_exact_without_norm(lib, page, d):
    b = Batch(RAGGED, 2, page, d, page + d, behind=3)
    cache = b.cache(lib)
    k, kx = bf16(b.rng, b.t, 2, d)
    v, vx = bf16(b.rng, b.t, 2, d, scale=2.0)
    assert lib.kv_update(cache, k, v, *b.args()) is None
    assert lib.get_device_error() == 0
    R.update(b.ref, kx, vx, b.table, b.start, b.kv_len)
    for got, ref in ((cache.k_scales, b.ref.scales[0]), (cache.v_scales, b.ref.scales[1]),
                     (cache.k_codes, b.ref.codes[0]), (cache.v_codes, b.ref.codes[1])):
        assert np.array_equal(got.cpu().numpy(), ref)     # spare pages and places behind the tokens among them


@pytest.mark.parametrize("page,d,hq,hk,rot,interleaved,given", [
    (16, 64, 4, 2, 64, False, False), (64, 128, 8, 8, 128, True, False), (32, 256, 6, 1, 64, False, True),
    (128, 128, 5, 1, 32, False, False)])
def test_update_with_norm_and_rotation(lib, page, d, hq, hk, rot, interleaved, given):
    b = Batch(RAGGED, hk, page, d, 7 * page + d, behind=2)
    cache = b.cache(lib)
    q, qx = bf16(b.rng, b.t, hq, d)
    k, kx = bf16(b.rng, b.t, hk, d)
    v, vx = bf16(b.rng, b.t, hk, d)
    qw, kw = (b.rng.random(d) + 0.5).astype(np.float32), (b.rng.random(d) + 0.5).astype(np.float32)
    pos = np.zeros(b.t, np.int32)
    for i, n in enumerate(b.q_len):
        pos[b.start[i]:b.start[i + 1]] = np.arange(b.kv_len[i] - n, b.kv_len[i])
    if given:
        pos = b.rng.integers(0, 200000, b.t).astype(np.int32)
    out = torch.full_like(q, -3.0)
    lib.kv_update(cache, k, v, *b.args(), q=q, q_out=out, positions=dev(pos) if given else None, q_weight=dev(qw),
                  k_weight=dev(kw), inv_freq=dev(INV[rot]), interleaved=interleaved)
    assert lib.get_device_error() == 0
    n = int(b.start[-1])
    check_heads(out[:n], R.norm_rope(qx, qw, 1e-6, pos, INV[rot], interleaved)[:n], pair_size(qx, qw, rot, interleaved, 1.0)[:n])
    assert (out[n:] == -3).all()                          # rows behind the last sequence
    R.update(b.ref, R.norm_rope(kx, kw, 1e-6, pos, INV[rot], interleaved), vx, b.table, b.start, b.kv_len)
    assert np.array_equal(cache.v_scales.cpu().numpy(), b.ref.scales[1])
    assert np.array_equal(cache.v_codes.cpu().numpy(), b.ref.codes[1])
    assert np.allclose(cache.k_scales.cpu().numpy(), b.ref.scales[0], rtol=2.0 ** -19)
    off = np.abs(cache.k_codes.cpu().numpy().astype(int) - b.ref.codes[0])
    assert off.max() <= 1 and (off > 0).mean() <= 3e-3


def test_update_scale_grows_stays_and_restarts(lib):
    """Token by token: recoding under a grown scale, none under a smaller value, a zero token, a reused page."""
    page, d = 16, 64
    b = Batch([(1, 1)], 1, page, d, 11)
    b.table = np.array([[2, 0, 1]], np.int32)
    cache = b.cache(lib)
    sizes = [1.0, 0.0, 5.0, 0.1, 30.0, 29.0] + [1.0] * 10 + [0.0, 3.0]
    for i, size in enumerate(sizes):
        k, kx = bf16(b.rng, 1, 1, d, scale=size)
        v, vx = bf16(b.rng, 1, 1, d, scale=size)
        kv = np.array([i + 1], np.int32)
        lib.kv_update(cache, k, v, dev(b.table), dev(np.array([0, 1], np.int32)), dev(kv))
        R.update(b.ref, kx, vx, b.table, [0, 1], kv)
    for got, ref in ((cache.k_scales, b.ref.scales[0]), (cache.k_codes, b.ref.codes[0]), (cache.v_codes, b.ref.codes[1])):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_dequant(lib):
    b = Batch([(1, 50)], 3, 32, 128, 12)
    cache = b.cache(lib)
    ids = np.array([3, 0, 3, 1], np.int32)
    for got, kind in zip(lib.kv_dequant(cache, dev(ids)), (0, 1)):
        ref = np.stack([[b.ref.values(kind, i, h) for h in range(3)] for i in ids])
        got = got.double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(ref))


# ---------------------------------------------------------------- attention

def check_attention(got, ref, absv, top, share, least=2.0 ** -39):
    live = ~np.isnan(ref)
    got = got.double().cpu().numpy()
    assert np.isfinite(got[live]).all()
    bar = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -16 + 2 * 2.0 ** -18 * top[..., None]) * absv
    bar = bar + least * 2.0 ** 7 * share[..., None] + 2.0 ** -73
    over = (np.abs(got - ref) - bar)[live]
    assert over.max() <= 0, f"{(over > 0).sum()} outputs off, worst {over.max():.3e}"


def attend(lib, b, hq, d, window=0, q_scale=1.0, least=2.0 ** -39):
    q, qx = bf16(b.rng, b.t, hq, d, scale=q_scale)
    out = torch.full_like(q, -3.0)
    lib.kv_attention(q, b.cache(lib), *b.args(), window=window, out=out)
    assert lib.get_device_error() == 0
    check_attention(out, *R.attention(qx, b.ref, b.table, b.start, b.kv_len, d ** -0.5, window), least=least)
    assert (out[int(b.start[-1]):] == -3).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attention_ragged(lib, page, d):
    attend(lib, Batch(RAGGED, 2, page, d, page * d, behind=2), 6, d)


@pytest.mark.parametrize("lens,hq,hk,page,d,window", [
    ([(1, 1)], 1, 1, 16, 64, 0),                       # one token
    ([(1, 2)], 1, 1, 16, 128, 0),
    ([(1, 255), (1, 256), (1, 257)], 24, 4, 64, 256, 0),
    ([(1, 3000)], 8, 1, 16, 128, 0),                   # one long sequence over many CTAs
    ([(1, 2500), (1, 70), (1, 1111)], 16, 16, 32, 64, 0),
    ([(1, 700), (3, 300)], 20, 1, 128, 128, 0),        # 20 heads to a key head: two row tiles
    ([(40, 200), (100, 100)], 4, 2, 32, 128, 0),       # many new tokens
    ([(130, 300)], 7, 1, 64, 64, 0),
    ([(1, 500), (20, 400), (9, 9)], 4, 2, 16, 128, 1),     # windows
    ([(1, 500), (20, 400), (9, 9)], 4, 2, 16, 128, 37),
    ([(60, 900)], 6, 2, 64, 256, 128),
    ([(1, 2000)], 6, 2, 32, 64, 500),
])
def test_attention_shapes(lib, lens, hq, hk, page, d, window):
    attend(lib, Batch(lens, hk, page, d, sum(a * b for a, b in lens) + d), hq, d, window)


@pytest.mark.parametrize("lens,hq,hk,page,d,window", [
    ([(256, 256)], 32, 32, 16, 128, 0),                # the rows of whole tiles, one group
    ([(200, 200), (150, 333), (1, 77)], 32, 16, 32, 128, 0),
    ([(129, 700), (3, 50), (260, 260)], 32, 16, 64, 64, 0),
    ([(150, 150), (0, 9), (135, 512)], 32, 16, 128, 256, 0),
    ([(70, 129), (128, 1000)], 64, 16, 16, 256, 0),
    ([(131, 640), (1, 5)], 56, 8, 16, 64, 0),          # seven heads to a key head
    ([(300, 900), (1, 300)], 16, 16, 16, 128, 100),    # windows, shorter and longer than a key tile
    ([(300, 900)], 16, 16, 32, 128, 1),
    ([(200, 700)], 16, 16, 64, 256, 260),
    ([(64, 2000)], 64, 32, 64, 128, 0),
])
def test_attention_many_new_tokens(lib, lens, hq, hk, page, d, window):
    """Sequences with enough rows for the tensor-memory kernel, alone and beside short ones."""
    attend(lib, Batch(lens, hk, page, d, sum(a * b for a, b in lens) + d + window, behind=2), hq, d, window,
           least=2.0 ** -32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_many_new_tokens_ranges(lib, d):
    """As the ranges below, on the tensor-memory kernel; a negative scale, which turns the order of the scores."""
    b = Batch([(130, 400), (140, 150)], 16, 16, d, d + 1)
    b.ref.scales[1][:] *= 10.0 ** b.rng.integers(-6, 7, b.ref.scales[1].shape)
    b.ref.scales[1][::3] = 0.0
    b.ref.scales[0][::4] = 0.0
    attend(lib, b, 16, d, q_scale=8.0, least=2.0 ** -32)
    q, _ = bf16(b.rng, b.t, 16, d)
    size = (10.0 ** b.rng.integers(-30, 3, (b.t, 16, 1))).astype(np.float32)
    q = (q.float() * dev(size)).to(torch.bfloat16)
    for scale in (d ** -0.5, -0.1):
        got = lib.kv_attention(q, b.cache(lib), *b.args(), scale=scale)
        check_attention(got, *R.attention(q.double().cpu().numpy(), b.ref, b.table, b.start, b.kv_len, scale),
                        least=2.0 ** -32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_ranges(lib, d):
    """Queries of far sizes (rows of 1e-30 to 1e30 within one tile), page scales from 0 to 1e6, sharp softmax."""
    b = Batch([(1, 400), (8, 90)], 2, 16, d, d)
    b.ref.scales[1][:] *= 10.0 ** b.rng.integers(-6, 7, b.ref.scales[1].shape)
    b.ref.scales[1][::3] = 0.0
    b.ref.scales[0][::4] = 0.0
    attend(lib, b, 4, d, q_scale=8.0)
    q, qx = bf16(b.rng, b.t, 4, d)
    size = (10.0 ** b.rng.integers(-30, 3, (b.t, 4, 1))).astype(np.float32)
    q = (q.float() * dev(size)).to(torch.bfloat16)
    got = lib.kv_attention(q, b.cache(lib), *b.args())
    check_attention(got, *R.attention(q.double().cpu().numpy(), b.ref, b.table, b.start, b.kv_len, d ** -0.5))


def test_attention_ignores_what_no_token_owns(lib):
    """Places behind a sequence's tokens hold extreme codes, pages behind them a NaN scale: nothing changes."""
    b = Batch([(1, 41), (1, 7)], 2, 16, 128, 30)
    q, _ = bf16(b.rng, b.t, 4, 128)
    cache = b.cache(lib)
    want = lib.kv_attention(q, cache, *b.args())
    for i, n in enumerate(b.kv_len):
        last = int(b.table[i, (n - 1) // 16])
        cache.k_codes[last, :, (n - 1) % 16 + 1:] = 127
        cache.v_codes[last, :, (n - 1) % 16 + 1:] = -128
    used = set(b.table[b.table >= 0].tolist())
    for i in range(b.pages):
        if i not in used:
            cache.k_scales[i], cache.v_scales[i] = float("nan"), float("nan")
    assert torch.equal(lib.kv_attention(q, cache, *b.args()), want)


def test_attention_is_repeatable_and_workspace_is_reusable(lib):
    """One workspace over shapes and replays; the same bits every time."""
    batches = [(Batch([(1, 3000), (1, 10), (1, 999)], 2, 16, 128, 40), 8, 128), (Batch(RAGGED, 1, 64, 256, 41), 6, 256),
               (Batch([(1, 2000)], 4, 32, 64, 42), 4, 64)]
    need = max(lib.kv_attention_workspace(b.t, hq, b.ref.scales[0].shape[1], d, "cuda").numel() for b, hq, d in batches)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = []
    for turn in range(3):
        for i, (b, hq, d) in enumerate(batches):
            if turn == 0:
                b.q, b.c = bf16(b.rng, b.t, hq, d)[0], b.cache(lib)
            got = lib.kv_attention(b.q, b.c, *b.args(), workspace=ws)
            if turn == 0:
                first.append(got)
                assert torch.equal(got, lib.kv_attention(b.q, b.c, *b.args()))
            assert torch.equal(got, first[i])
    assert not ws[:1024].any()


def test_bad_numbers_are_reported_and_left_out(lib):
    """Page ids and lengths outside the buffers: the call reports them, other sequences are unharmed."""
    b = Batch([(1, 40), (1, 30), (1, 50)], 2, 16, 128, 50)
    q, qx = bf16(b.rng, b.t, 4, 128)
    cache = b.cache(lib)
    table, start, kv = b.args()
    want = lib.kv_attention(q, cache, table, start, kv)
    k, _ = bf16(b.rng, b.t, 2, 128)
    for bad in (b.pages, -5, 2 ** 31 - 1):
        broken = table.clone()
        broken[1, 1] = bad
        got = lib.kv_attention(q, cache, broken, start, kv)
        assert lib.get_device_error() == 8                # W4A8_ERR_INPUT
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        before = cache.k_codes.clone()
        lib.kv_update(cache, k, k, broken, start, kv)
        assert lib.get_device_error() == 8
        assert torch.equal(cache.k_codes[int(b.table[1, 1])], before[int(b.table[1, 1])])
        cache = b.cache(lib)
    for wrong in ((kv, torch.tensor([40, 1000, 50], dtype=torch.int32, device="cuda")),
                  (kv, torch.tensor([40, 0, 50], dtype=torch.int32, device="cuda"))):
        got = lib.kv_attention(q, cache, table, start, wrong[1], out=torch.full_like(q, -3.0))
        assert lib.get_device_error() == 8
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and (got[1] == -3).all()
    got = lib.kv_attention(q, cache, table, torch.tensor([0, 1, 2, 9], dtype=torch.int32, device="cuda"), kv)
    assert lib.get_device_error() == 8 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ids = torch.tensor([0, b.pages, -1], dtype=torch.int32, device="cuda")
    vals, _ = lib.kv_dequant(cache, ids)
    assert lib.get_device_error() == 8 and not vals[1:].any() and vals[0].any()
    assert lib.get_device_error() == 0


def test_decode_steps_together(lib):
    """A conversation as it is used: a chunk, then token by token, each step the update and the attention, against
    the oracle's cache after the same steps; captured steps replay to the same bits."""
    page, d, hq, hk = 16, 128, 8, 2
    b = Batch([(37, 37), (20, 20)], hk, page, d, 60, spare=8)
    b.table = np.array([[1, 2, 3, 4], [5, 6, 7, 8]], np.int32)
    cache = b.cache(lib)
    kw, inv = dev(np.ones(d, np.float32)), dev(INV[128])
    lens = np.array([0, 0], np.int32)
    for step, new in enumerate([(37, 20)] + [(1, 1)] * 14):
        n = np.array(new, np.int32)
        lens = lens + n
        start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        t = int(n.sum())
        q, qx = bf16(b.rng, t, hq, d)
        k, kx = bf16(b.rng, t, hk, d)
        v, vx = bf16(b.rng, t, hk, d)
        idx = dev(b.table), dev(start), dev(lens)
        qo = lib.kv_update(cache, k, v, *idx, q=q, q_weight=kw, k_weight=kw, inv_freq=inv)
        out = lib.kv_attention(qo, cache, *idx)
        if step in (0, 1, 7, 14):
            now = R.Cache(*(a.cpu().numpy() for a in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)))
            check_attention(out, *R.attention(qo.double().cpu().numpy(), now, b.table, start, lens, d ** -0.5))
    g = torch.cuda.CUDAGraph()
    ws = lib.kv_attention_workspace(t, hq, hk, d, "cuda")
    again = torch.zeros_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        lib.kv_update(cache, k, v, *idx, q=q, q_weight=kw, k_weight=kw, inv_freq=inv, q_out=qo)
        lib.kv_attention(qo, cache, *idx, workspace=ws, out=again)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out) and lib.get_device_error() == 0


@pytest.mark.parametrize("lens", [[(1, 300), (1, 16)], [(150, 700), (64, 64)]])
@pytest.mark.parametrize("scale,window", [(0.0, 0), (0.0, 5), (0.3, 1)])
def test_attention_even_and_single(lib, lens, scale, window):
    """A scale of zero (the mean of the values), and a window of one token (its own value), of few and of many rows."""
    b = Batch(lens, 4, 16, 128, 70)
    q, qx = bf16(b.rng, b.t, 32, 128)
    out = lib.kv_attention(q, b.cache(lib), *b.args(), scale=scale, window=window)
    assert lib.get_device_error() == 0
    check_attention(out, *R.attention(qx, b.ref, b.table, b.start, b.kv_len, scale, window), least=2.0 ** -32)


def test_rows_before_the_first_sequence(lib):
    """q_start[0] > 0: the rows before it are no sequence's, and stay as they were."""
    b = Batch([(2, 40), (1, 30)], 2, 16, 128, 71)
    pad = lambda x: torch.cat([torch.full_like(x[:2], 9.0), x])
    q, k, v = (bf16(b.rng, b.t, h, 128)[0] for h in (4, 2, 2))
    table, start, kv = b.args()
    kw, inv = dev(np.ones(128, np.float32)), dev(INV[128])
    one, two = b.cache(lib), b.cache(lib)
    qo = lib.kv_update(one, k, v, table, start, kv, q=q, q_weight=kw, k_weight=kw, inv_freq=inv, q_out=torch.full_like(q, -3.0))
    want = lib.kv_attention(qo, one, table, start, kv, out=torch.full_like(q, -3.0))
    qp = lib.kv_update(two, pad(k), pad(v), table, start + 2, kv, q=pad(q), q_weight=kw, k_weight=kw, inv_freq=inv,
                       q_out=torch.full_like(pad(q), -3.0))
    got = lib.kv_attention(qp, two, table, start + 2, kv, out=torch.full_like(pad(q), -3.0))
    assert lib.get_device_error() == 0
    assert torch.equal(qp[2:], qo) and torch.equal(got[2:], want)
    assert (qp[:2] == -3).all() and (got[:2] == -3).all()
    assert torch.equal(one.k_codes, two.k_codes) and torch.equal(one.v_scales, two.v_scales)


def test_calls_on_another_stream(lib):
    """A stream given by name, with the current one behind: the call waits for nothing of it, its own workspace
    included, and gives the same bits."""
    b = Batch([(1, 3000), (1, 70), (300, 400)], 2, 16, 128, 72)
    q, _ = bf16(b.rng, b.t, 8, 128)
    k, _ = bf16(b.rng, b.t, 2, 128)
    kw, inv = dev(np.ones(128, np.float32)), dev(INV[128])
    pos = torch.arange(b.t, dtype=torch.int32, device="cuda")
    ids = torch.arange(b.pages, dtype=torch.int32, device="cuda")
    def run(cache, stream):
        qo, _ = lib.qk_norm_rope(q, None, pos, kw, None, inv_freq=inv, stream=stream)
        qo = lib.kv_update(cache, k, k, *args, q=qo, k_weight=kw, inv_freq=inv, stream=stream)
        return [qo, lib.kv_attention(qo, cache, *args, stream=stream), *lib.kv_dequant(cache, ids, stream=stream)]
    args, one, two = b.args(), b.cache(lib), b.cache(lib)
    want = run(one, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    got = run(two, s)
    s.synchronize()
    assert lib.get_device_error() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_cache_is_what_it_holds_at_the_call(lib):
    """Tensors put into a cache after it was made are the ones that the next call reads."""
    b = Batch([(1, 40), (1, 7)], 2, 16, 128, 73)
    q, _ = bf16(b.rng, b.t, 4, 128)
    one, two = b.cache(lib), b.cache(lib)
    two.k_codes.zero_()
    two.v_scales.mul_(2)
    want = lib.kv_attention(q, two, *b.args())
    one.k_codes, one.v_scales = two.k_codes, two.v_scales
    assert torch.equal(lib.kv_attention(q, one, *b.args()), want)
    for name, bad in (("k_codes", two.k_codes[1:]), ("v_codes", two.v_codes.float()), ("k_scales", two.k_scales.cpu()),
                      ("v_scales", None)):
        broken = b.cache(lib)
        setattr(broken, name, bad)
        with pytest.raises(ValueError):
            lib.kv_attention(q, broken, *b.args())
        with pytest.raises(ValueError):
            lib.kv_update(broken, q[:, :2], q[:, :2], *b.args())


def test_refused_before_anything_runs(lib):
    """A number that is none leaves the cache as it was; heads whose size does not fit 32 bits are not cut to it."""
    b = Batch([(1, 40), (1, 7)], 2, 16, 128, 74)
    k, _ = bf16(b.rng, b.t, 2, 128)
    cache = b.cache(lib)
    before = cache.k_codes.clone()
    for bad in (dict(eps="small"), dict(eps=None), dict(rope_factor="one", inv_freq=dev(INV[128]))):
        with pytest.raises(TypeError):
            lib.kv_update(cache, k, k, *b.args(), k_weight=dev(np.ones(128, np.float32)), **bad)
    with pytest.raises(TypeError):
        lib.kv_attention(k, cache, *b.args(), scale="one")
    for bad in (-1, 2 ** 40):
        with pytest.raises(ValueError):
            lib.kv_attention(k, cache, *b.args(), window=bad)
    torch.cuda.synchronize()
    assert torch.equal(cache.k_codes, before)
    wide = torch.empty((1, 1, 2 ** 32 + 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        lib.qk_norm_rope(wide, None, q_out=wide)
    shared = torch.empty((1, 4, 128), dtype=torch.bfloat16, device="cuda").expand(b.t, 4, 128)
    with pytest.raises(lib.W4A8Error):
        lib.kv_attention(torch.zeros(b.t, 4, 128, dtype=torch.bfloat16, device="cuda"), cache, *b.args(), out=shared)


@pytest.mark.parametrize("lens,hq,hk,page,d,window", [
    ([(700, 1500)], 32, 8, 32, 128, 0),                       # less than a wave of tiles: all in parts
    ([(130, 130), (64, 6000), (200, 1000)], 16, 4, 64, 64, 0),  # parts of very different ranges
    ([(1300, 2000), (900, 900)], 32, 8, 16, 128, 300),        # a wave and a rest; the window leaves most keys out
    ([(1024, 1100)], 24, 4, 64, 256, 0),
    ([(1, 5), (1, 4)], 1024, 8, 16, 64, 0),                   # one tile of keys: parts without any
    ([(1, 80)] * 5, 2048, 16, 16, 128, 0),
])
def test_attention_parts(lib, lens, hq, hk, page, d, window):
    """Row tiles split along their keys: against the oracle, the same bits again, and a clean workspace."""
    b = Batch(lens, hk, page, d, 75)
    q, qx = bf16(b.rng, b.t, hq, d)
    cache, ws = b.cache(lib), lib.kv_attention_workspace(b.t, hq, hk, d, "cuda")
    out = lib.kv_attention(q, cache, *b.args(), window=window, workspace=ws)
    assert lib.get_device_error() == 0
    check_attention(out, *R.attention(qx, b.ref, b.table, b.start, b.kv_len, d ** -0.5, window), least=2.0 ** -32)
    assert not ws[:1024].any()
    ws[1024:] = 255                                           # (NaN in every partial result that is not written)
    for _ in range(3):
        assert torch.equal(lib.kv_attention(q, cache, *b.args(), window=window, workspace=ws), out)
    assert not ws[:1024].any()


def test_sequences_that_share_rows_leave_the_workspace_clean(lib):
    """q_start that goes back and forth: results are undefined, the next call's are not."""
    b = Batch([(700, 1500)], 8, 32, 128, 76)
    q, _ = bf16(b.rng, b.t, 32, 128)
    cache, ws = b.cache(lib), lib.kv_attention_workspace(b.t, 32, 8, 128, "cuda")
    want = lib.kv_attention(q, cache, *b.args(), workspace=ws)
    table, _, kv = b.args()
    start = torch.tensor([0, b.t] * 5, dtype=torch.int32, device="cuda")
    lib.kv_attention(q, cache, table.repeat(9, 1), start, kv.repeat(9), workspace=ws)
    assert lib.get_device_error() == 8
    assert not ws[:1024].any()
    assert torch.equal(lib.kv_attention(q, cache, *b.args(), workspace=ws), want)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(8, 2), (24, 4), (7, 1), (12, 1), (16, 16)])
def test_attention_row_tiles(lib, d, hq, hk):
    """Row tiles of 8 that a sequence fills in part, once and several times, among empty sequences; groups that do
    not divide 8, and one of more rows than 8."""
    b = Batch([(5, 40), (0, 9), (0, 0), (3, 1000), (0, 70), (1, 1), (0, 16), (1, 333)], hk, 32, d, 77, behind=2)
    attend(lib, b, hq, d)
    attend(lib, b, hq, d, window=20)


@pytest.mark.parametrize("lens,hq,hk,page,d,window", [
    ([(256, 3000)], 32, 32, 16, 128, 0),
    ([(200, 2200), (150, 3333), (1, 77)], 32, 16, 32, 128, 0),
    ([(129, 2700), (3, 50), (260, 2600)], 32, 16, 64, 64, 0),
    ([(150, 3150), (0, 9), (135, 2512)], 32, 16, 128, 256, 0),
    ([(70, 3129), (128, 1000)], 64, 16, 16, 256, 0),
    ([(131, 3640), (1, 5)], 56, 8, 16, 64, 0),
    ([(700, 900)], 64, 16, 32, 128, 1),
    ([(600, 1700)], 32, 16, 64, 256, 260),
    ([(130, 130), (128, 6000), (200, 1000)], 16, 4, 64, 128, 0),
    ([(400, 6000), (32, 32)], 16, 4, 64, 128, 0),      # parts of a unit with one tile of keys
])
def test_attention_many_rows_and_keys(lib, lens, hq, hk, page, d, window):
    """Batches whose rows and keys pay for the tensor-memory kernel (kv_tiles_pay), alone and beside short ones."""
    attend(lib, Batch(lens, hk, page, d, 78 + d + window, behind=2), hq, d, window, least=2.0 ** -32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_many_rows_and_keys_ranges(lib, d):
    """Page scales from 0 to 1e6, queries of far sizes, a negative scale, on the tensor-memory kernel."""
    b = Batch([(130, 3000), (140, 2150)], 16, 16, d, d + 2)
    b.ref.scales[1][:] *= 10.0 ** b.rng.integers(-6, 7, b.ref.scales[1].shape)
    b.ref.scales[1][::3] = 0.0
    b.ref.scales[0][::4] = 0.0
    attend(lib, b, 32, d, q_scale=8.0, least=2.0 ** -32)
    q, _ = bf16(b.rng, b.t, 32, d)
    size = (10.0 ** b.rng.integers(-30, 3, (b.t, 32, 1))).astype(np.float32)
    q = (q.float() * dev(size)).to(torch.bfloat16)
    got = lib.kv_attention(q, b.cache(lib), *b.args(), scale=-0.1)
    check_attention(got, *R.attention(q.double().cpu().numpy(), b.ref, b.table, b.start, b.kv_len, -0.1), least=2.0 ** -32)
