"""GPU parity of the int8 layer (w4a8_int8_* of include/w4a8_int8.h) against
oracle/int8_ref.py.

Bars:
  * quantiser without rotation: bit-exact (every decision is an fp32
    operation on the same inputs); with rotation: the codes and scales of
    w4a8_rotate_quant_act, bit for bit, and against the oracle at most one
    step on at most 1e-3 of the codes (the fp32 butterflies put a value within
    127 * 2^-20 of a step off its fp64 place: 2.4e-4 of them may change);
  * product: the integer sum is exact, its conversion and the two scalings
    round in fp32 (2^-24 each), the result to bf16 (half a step: 2^-8):
    |y - ref| <= (2^-8 + 2^-22) |ref|;
  * layer: the product on the codes that the quantiser gave.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import int8_ref as R

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(bits):
    return dev(bits.view(np.int16)).view(torch.bfloat16)


def acts(m, k, seed):
    bits, x, _ = synth.activations(m, k, synth.rng_for(seed, m, "act"), max(1, k // 100))
    return bits, x


def check(y, ref):
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    over = np.abs(y - ref) - (2.0 ** -8 + 2.0 ** -22) * np.abs(ref)
    assert over.max() <= 0, f"{(over > 0).sum()} outputs off, worst {over.max():.3e}"


@pytest.mark.parametrize("r,k", [(1, 16), (3, 48), (5, 272), (2, 4304), (4, 8192), (300, 528), (2, 32768)])
@pytest.mark.parametrize("f32", [False, True])
def test_quantize_without_rotation_is_exact(lib, r, k, f32):
    bits, x = acts(r, k, 70)
    x = x.copy()
    if r > 1:
        x[1] = 0                                   # a row of zeros
        bits[1] = 0
    codes, s = lib.int8_quantize(dev(x) if f32 else bf16(bits), rotate=False)
    ref_codes, ref_s = R.quantize_rows(x, rotate=False)
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(codes.cpu().numpy(), ref_codes)


@pytest.mark.parametrize("r,k", [(1, 256), (3, 512), (40, 5120), (297, 768), (2, 17408)])
def test_quantize_with_rotation(lib, r, k):
    bits, x = acts(r, k, 71)
    codes, s = lib.int8_quantize(bf16(bits), rotate=True)
    same_codes, same_s = lib.rotate_quant_act(bf16(bits))
    assert torch.equal(codes, same_codes) and torch.equal(s, same_s)
    ref_codes, ref_s = R.quantize_rows(x, rotate=True)
    assert np.allclose(s.cpu().numpy(), ref_s, rtol=2.0 ** -20)
    off = np.abs(codes.cpu().numpy().astype(int) - ref_codes)
    assert off.max() <= 1 and (off > 0).sum() <= max(2, 1e-3 * off.size)
    w = synth.weights(r, k, synth.rng_for(72, r, "weight"))
    c32, _ = lib.int8_quantize(dev(w), rotate=True)
    off = np.abs(c32.cpu().numpy().astype(int) - R.quantize_rows(w, rotate=True)[0])
    assert off.max() <= 1 and (off > 0).sum() <= max(2, 1e-3 * off.size)


def operands(m, n, k, seed):
    rng = np.random.default_rng(seed)
    x = rng.integers(-127, 128, (m, k), dtype=np.int8)
    w = rng.integers(-127, 128, (n, k), dtype=np.int8)
    return x, (rng.random(m, np.float32) + 0.1), w, (rng.random(n, np.float32) + 0.1)


SHAPES = [
    (1, 1, 16),            # the smallest
    (1, 128, 128),         # one tile, one k block
    (4, 256, 512),
    (16, 130, 272),        # k past a block, a second row tile of two rows
    (17, 100, 4304),
    (31, 1000, 144),
    (64, 257, 1024),
    (65, 129, 640),
    (128, 384, 256),
    (129, 255, 400),       # 256-token tiles, ragged everywhere
    (300, 200, 1280),
    (513, 136, 2560),      # the last token tile holds one token
    (1, 5120, 5120),       # tiles cut between CTAs
    (50, 1161, 4304),
    (2048, 2048, 256),     # whole 256 x 256 tiles on pairs of CTAs, two k blocks
    (2000, 2300, 400),     # ragged tokens, rows and k; rows of y 8-byte aligned only
    (1025, 6001, 1040),    # one token in the last tile, odd N
    (4097, 1100, 144),
]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(lib, m, n, k):
    x, sx, w, sw = operands(m, n, k, m + n + k)
    y = lib.int8_gemm(dev(x), dev(sx), dev(w), dev(sw))
    assert lib.get_device_error() == 0
    check(y, R.product(x, sx, w, sw))


def test_product_extremes(lib):
    """Codes of -128, the largest K, and rows whose scale is 0."""
    m, n, k = 3, 130, 32768
    x, w = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    w[1::2] = 127
    sx, sw = np.array([1e-3, 0.0, 2.0], np.float32), np.full(n, 0.5, np.float32)
    y = lib.int8_gemm(dev(x), dev(sx), dev(w), dev(sw))
    check(y, R.product(x, sx, w, sw))
    assert not y[1].any()


def test_one_workspace_serves_every_shape(lib):
    """Layers of different shapes on one workspace, in turn, whatever it held before."""
    shapes = [(1, 592, 768), (300, 200, 1280), (45, 1000, 512), (1, 592, 768)]
    ws = torch.full((max(lib.int8_linear_workspace(m, k, n, "cuda").numel() for m, n, k in shapes),), 255,
                    dtype=torch.uint8, device="cuda")
    for m, n, k in shapes:
        bits, _ = acts(m, k, 75)
        wq, sw = lib.int8_quantize(dev(synth.weights(n, k, synth.rng_for(75, n, "weight"))))
        xq, sx = lib.int8_quantize(bf16(bits))
        check(lib.int8_linear(bf16(bits), wq, sw, workspace=ws), R.product(*(t.cpu().numpy() for t in (xq, sx, wq, sw))))


@pytest.mark.parametrize("m,n,k,rotate", [(1, 592, 768, True), (1, 300, 4304, False), (7, 130, 512, True),
                                          (45, 1000, 4304, False), (200, 384, 1024, True), (600, 200, 528, False)])
def test_layer(lib, m, n, k, rotate):
    bits, x = acts(m, k, 73)
    w = synth.weights(n, k, synth.rng_for(73, n, "weight"))
    wq, sw = lib.int8_quantize(dev(w), rotate=rotate)
    xq, sx = lib.int8_quantize(bf16(bits), rotate=rotate)
    y = lib.int8_linear(bf16(bits), wq, sw, rotate=rotate)
    assert lib.get_device_error() == 0
    check(y, R.product(*(t.cpu().numpy() for t in (xq, sx, wq, sw))))
    # and it is x W^T: with |x - x^| <= s_x / 2 and |w - w^| <= s_w / 2 (half a step of each code, in the rotated
    # basis where rotated, which leaves the product as it is), every output is within
    # s_x / 2 sum |w^| + s_w / 2 sum |x^| + K s_x s_w / 4 of it, plus bf16's 2^-8 and the fp32 rotation's 2^-19
    xh, wh = (c.double().cpu().numpy() * s.double().cpu().numpy()[:, None] for c, s in ((xq, sx), (wq, sw)))
    sx, sw = sx.double().cpu().numpy()[:, None], sw.double().cpu().numpy()[None, :]
    bar = sx / 2 * np.abs(wh).sum(1)[None, :] + sw / 2 * np.abs(xh).sum(1)[:, None] + k * sx * sw / 4
    ref = x.astype(np.float64) @ w.astype(np.float64).T
    size = np.abs(xh) @ np.abs(wh).T
    got = y.double().cpu().numpy()
    assert (np.abs(got - ref) <= bar + 2.0 ** -8 * np.abs(got) + 2.0 ** -19 * (size + bar)).all()


def test_out_stays_inside(lib):
    """Guard bands around y survive (ragged rows and tokens)."""
    for m, n, k in ((3, 37, 64), (130, 131, 144)):
        x, sx, w, sw = operands(m, n, k, 5)
        buf = torch.full((64 + m * n + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
        lib.int8_gemm(dev(x), dev(sx), dev(w), dev(sw), out=buf[64:64 + m * n].view(m, n))
        assert (buf[:64] == -7).all() and (buf[64 + m * n:] == -7).all()
        check(buf[64:64 + m * n].view(m, n), R.product(x, sx, w, sw))


def test_captured_and_replayed_on_another_stream(lib):
    m, n, k = 5, 1000, 4096
    bits, _ = acts(m, k, 74)
    w = synth.weights(n, k, synth.rng_for(74, n, "weight"))
    wq, sw = lib.int8_quantize(dev(w), rotate=True)
    x = bf16(bits)
    want = lib.int8_linear(x, wq, sw)
    ws = lib.int8_linear_workspace(m, k, n, "cuda")
    out = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                lib.int8_linear(x, wq, sw, workspace=ws, out=out)
        for _ in range(4):
            out.zero_()
            g.replay()
    s.synchronize()
    assert torch.equal(out, want)


def test_refusals_of_the_binding(lib):
    x = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    w, s = torch.zeros(64, 512, dtype=torch.int8, device="cuda"), torch.zeros(64, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:, ::2]), dict(w=w.float()), dict(w=w[:, :256].contiguous()), dict(s=s[:10].contiguous()),
                dict(s=s.double()), dict(out=torch.zeros(4, 63, dtype=torch.bfloat16, device="cuda"))):
        a = {"x": x, "w": w, "s": s, "out": None, **bad}
        with pytest.raises(ValueError):
            lib.int8_linear(a["x"], a["w"], a["s"], out=a["out"])
    with pytest.raises(lib.W4A8Error):
        lib.int8_linear(x, w, s, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.W4A8Error):
        lib.int8_linear(x[:, :272].contiguous(), w[:, :272].contiguous(), s, rotate=True)


def test_weights_quantised_just_before_the_product(lib):
    """The product fetches weights ahead of the kernel before it; one that writes them must have completed."""
    m, n, k = 4, 464, 16384   # rows of the quantiser: a last wave of a few of the 148 SMs
    x, sx, _, _ = operands(m, 16, k, 6)
    x, sx = dev(x), dev(sx)
    w = torch.randn(n, k, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    codes, s = lib.int8_quantize(w, rotate=False)
    torch.cuda.synchronize()
    want = lib.int8_gemm(x, sx, codes, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            old = torch.full((n, k), 77, dtype=torch.int8, device="cuda")  # what the next allocation finds in its place
            del old
            wq, sw = lib.int8_quantize(w, rotate=False)
            y = lib.int8_gemm(x, sx, wq, sw)
            del wq, sw
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_scratch_belongs_to_the_calls_stream(lib):
    """Without a workspace, on another stream that is behind: what the current stream allocates meanwhile is not it."""
    m, n, k = 200, 1000, 4096
    bits, _ = acts(m, k, 75)
    wq, sw = lib.int8_quantize(dev(synth.weights(n, k, synth.rng_for(75, n, "weight"))), rotate=True)
    x = bf16(bits)
    want = lib.int8_linear(x, wq, sw)
    s = torch.cuda.Stream()
    torch.full((8,), 77, dtype=torch.uint8, device="cuda")  # (a kernel's first launch may wait for the device)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    got = lib.int8_linear(x, wq, sw, stream=s)
    used = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for size in [m * k + 1024] * 4 + [m * n * 2] * 4]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all((u == 77).all() for u in used)


@pytest.mark.parametrize("r,k,rotate,f32", [(300, 16, False, False), (400, 17408, True, False), (297, 32768, True, False),
                                            (301, 4304, False, False), (500, 2304, True, True), (1000, 256, True, False),
                                            (298, 32752, False, True)])
def test_many_rows_are_the_few(lib, r, k, rotate, f32):
    """The kernel of many rows gives each row the codes and scale that the one of few rows gives it."""
    x = torch.randn(r, k, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
    x *= 10.0 ** torch.randint(-20, 20, (r, 1), device="cuda").float()
    x[3] = 0
    x = x if f32 else x.to(torch.bfloat16)
    codes, s = lib.int8_quantize(x, rotate=rotate)
    parts = [lib.int8_quantize(x[i:i + 200].contiguous(), rotate=rotate) for i in range(0, r, 200)]
    assert torch.equal(codes, torch.cat([c for c, _ in parts])) and torch.equal(s, torch.cat([t for _, t in parts]))
