"""AttentionBlock: the 8-bit path and the codebook layer as they are used
together.  Its output must be, bit for bit, what the separate calls give, for a
prompt and the tokens after it, eager and captured; and the attention that it
feeds the output projection must be the oracle's over the cache it has
written (the bars of test_gpu_kv.py: bf16 output 2^-8, fp16 weights 2^-11,
scores 2^-18)."""

import numpy as np
import pytest
import torch

import oracle as O
import synth
from oracle import int8_ref as R

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, D, PAGE = 768, 6, 2, 128, 16


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def codebook_layer(lib, n, k, seed):
    from w4a8_codebook_quantized_rotate_b200 import blocks
    c = O.convert_weight(synth.weights(n, k, synth.rng_for(seed, 0, "weight")))
    return blocks.CodebookLayer(lib.pack_layout(dev(c["packed"]), dev(c["s_rel"]), dev(c["s_ch"]), dev(c["cb"])), n, k)


def int8_layer(lib, n, k, seed):
    from w4a8_codebook_quantized_rotate_b200 import blocks
    return blocks.Int8Layer(*lib.int8_quantize(dev(synth.weights(n, k, synth.rng_for(seed, 1, "weight"))), rotate=True), rotate=True)


@pytest.fixture(params=["codebook qkv, int8 out", "int8 qkv, codebook out"])
def block(lib, request):
    from w4a8_codebook_quantized_rotate_b200 import blocks
    first = request.param.startswith("codebook")
    n = (HEADS + 2 * KV) * D
    qkv = (codebook_layer if first else int8_layer)(lib, n, HIDDEN, 80)
    out = (int8_layer if first else codebook_layer)(lib, HIDDEN, HEADS * D, 81)
    w = dev((np.random.default_rng(0).random(D) + 0.5).astype(np.float32))
    inv, factor = lib.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=32)
    return blocks.AttentionBlock(qkv, out, HEADS, KV, D, q_weight=w, k_weight=w, inv_freq=inv, rope_factor=factor)


def steps():
    lens = np.zeros(2, np.int32)
    for new in [(21, 40), (1, 1), (1, 1), (3, 0), (1, 1)]:
        lens = lens + np.array(new, np.int32)
        yield new, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), lens.copy()


def test_block_is_its_calls(lib, block):
    table = dev(np.array([[5, 1, 3, 7, 0], [2, 4, 6, 8, 9]], np.int32))
    one, two = (lib.KvCache(10, KV, PAGE, D) for _ in range(2))
    rng = synth.rng_for(82, 0, "act")
    r = block.rotation
    for new, start, lens in steps():
        t = int(sum(new))
        bits, _, _ = synth.activations(t, HIDDEN, rng, 8)
        x = dev(bits.view(np.int16)).view(torch.bfloat16)
        idx = table, dev(start), dev(lens)
        y = block(x, one, *idx)
        rows = block.qkv(x).view(t, HEADS + 2 * KV, D)
        q = lib.kv_update(two, rows[:, HEADS:HEADS + KV], rows[:, HEADS + KV:], *idx, q=rows[:, :HEADS], **r)
        o = lib.kv_attention(q, two, *idx)
        assert torch.equal(y, block.out(o.view(t, HEADS * D)))
        for a, b in ((one.k_codes, two.k_codes), (one.v_codes, two.v_codes), (one.k_scales, two.k_scales)):
            assert torch.equal(a, b)
        now = R.Cache(*(a.cpu().numpy() for a in (two.k_codes, two.v_codes, two.k_scales, two.v_scales)))
        ref, absv, top, share = R.attention(q.double().cpu().numpy(), now, table.cpu().numpy(), start, lens, D ** -0.5)
        bar = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -16 + 2.0 ** -17 * top[..., None]) * absv + 2.0 ** -32 * share[..., None]
        assert (np.abs(o.double().cpu().numpy() - ref) <= bar).all()
    assert lib.get_device_error() == 0


def test_block_step_captured(lib, block):
    """A decode step in a graph: replays read the lengths on the GPU, so one graph serves step after step."""
    table = dev(np.array([[5, 1, 3], [2, 4, 6]], np.int32))
    eager, graphed = (lib.KvCache(10, KV, PAGE, D) for _ in range(2))
    bits, _, _ = synth.activations(12, HIDDEN, synth.rng_for(83, 0, "act"), 8)
    xs = dev(bits.view(np.int16)).view(torch.bfloat16).view(6, 2, HIDDEN)
    start = dev(np.array([0, 1, 2], np.int32))
    want = [block(xs[i], eager, table, start, dev(np.array([i + 1, i + 1], np.int32))) for i in range(6)]
    block.prepare(2)
    x, lens = torch.zeros_like(xs[0]), torch.ones(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = block(x, graphed, table, start, lens)
    for i in range(6):
        x.copy_(xs[i])
        lens.fill_(i + 1)
        g.replay()
        assert torch.equal(y, want[i]), i
    assert torch.equal(eager.k_codes, graphed.k_codes) and lib.get_device_error() == 0


def test_block_refuses_layers_that_do_not_fit(lib, block):
    from w4a8_codebook_quantized_rotate_b200 import blocks
    with pytest.raises(ValueError):
        blocks.AttentionBlock(block.qkv, block.out, HEADS + 1, KV, D)
    with pytest.raises(ValueError):
        blocks.AttentionBlock(block.qkv, blocks.CodebookLayer(block.qkv, HIDDEN, 512), HEADS, KV, D)   # 512 inputs


def test_workspaces_serve_many_token_counts(lib):
    """Token counts up and down: a few workspaces serve them all, and every result is that of a fresh layer."""
    from w4a8_codebook_quantized_rotate_b200 import blocks
    for make in (codebook_layer, int8_layer):
        layer = make(lib, 320, 768, 83)
        x = torch.randn(300, 768, device="cuda", generator=torch.Generator("cuda").manual_seed(83)).to(torch.bfloat16)
        for m in (1, 300, 2, 7, 33, 129, 300, 64, 1, 257):
            fresh = (blocks.CodebookLayer(layer.packed, 320, 768) if make is codebook_layer
                     else blocks.Int8Layer(layer.w_q, layer.s_w, layer.rotate))
            assert torch.equal(layer(x[:m]), fresh(x[:m]))
        held = [w.numel() for w in layer._workspaces._held]
        assert all(b >= 2 * a for a, b in zip(held, held[1:])) and len(held) < 16
