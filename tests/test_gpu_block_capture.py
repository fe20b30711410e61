"""AttentionBlock in a capture that nothing was prepared for: refused, and the block works on as before."""

import pytest
import torch

from test_gpu_block import HIDDEN, KV, D, PAGE, block, dev  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_capture_without_workspaces_is_refused(lib, block):  # noqa: F811
    cache = [lib.KvCache(10, KV, PAGE, D) for _ in range(2)]
    table, start, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([[5, 1], [2, 4]], [0, 1, 2], [1, 1]))
    x = torch.randn(2, HIDDEN, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="prepare"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            block(x, cache[0], table, start, lens)
    want = block(x, cache[0], table, start, lens)            # its first eager step; then a capture is accepted
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = block(x, cache[1], table, start, lens)
    again = block(x, cache[0], table, start, lens)           # on the same workspaces, before the first replay
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(again, want) and lib.get_device_error() == 0
