"""Order on the GPU between the calls that make int8 weights and the product
that fetches them ahead of the kernel before it (include/w4a8_int8.h): every
call of the library that writes int8 codes must have completed by then."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layer", [False, True])
def test_weights_of_the_activation_quantiser_just_before_the_product(lib, layer):
    """bf16 weights quantised by rotate_quant_act, which gives the codes of int8_quantize, directly before int8_gemm,
    and before int8_linear (whose own quantiser stands between, but lets the product start early)."""
    m, n, k = 4, 464, 16384   # rows of the quantiser: a last wave of a few of the 148 SMs
    gen = torch.Generator("cuda").manual_seed(7)
    x = torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16)
    w = torch.randn(n, k, device="cuda", generator=gen).to(torch.bfloat16)
    xq, sx = lib.int8_quantize(x, rotate=True)
    codes, s = lib.int8_quantize(w, rotate=True)
    ws, out = lib.int8_linear_workspace(m, k, n, "cuda"), torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    want = lib.int8_gemm(xq, sx, codes, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            old = torch.full((n, k), 77, dtype=torch.int8, device="cuda")  # what the next allocation finds in its place
            del old
            wq, sw = lib.rotate_quant_act(w)
            if layer:
                lib.int8_linear(x, wq, sw, workspace=ws, out=out)
            else:
                lib.int8_gemm(xq, sx, wq, sw, out=out)
            del wq, sw
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
