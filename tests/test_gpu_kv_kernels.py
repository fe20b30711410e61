"""Attention over the int8 paged cache, each case on the kernel that it is
meant for: the choice (csrc/kv_index.h, compiled for the host) is asserted, and
the streaming kernel's cases hold its bar, 2^-39 of the largest share (bars of
test_gpu_kv.py; 2^-32 for the tensor-memory kernel)."""

import numpy as np
import pytest
import torch

import kv_index
import test_gpu_kv as T
import test_gpu_kv_edges as E
from oracle import int8_ref as R
from test_gpu_kv import Batch, attend, bf16, check_attention

pytestmark = pytest.mark.gpu

STREAM, TENSOR = 2.0 ** -39, 2.0 ** -32


def kernel(b, hq, hk, page, d, window=0):
    """The bar of the kernel that a batch runs on (with a tile of rows or more; short sequences beside it are streamed)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = [(n, int(kv)) for n, kv in zip(b.q_len, b.kv_len)]
    assert b.table.shape[1] == max(-(-n // page) for _, n in lens) + 1
    return TENSOR if kv_index.tensor_units(lens, hq, hk, page, d, window, b.t - int(b.start[-1]), sms) else STREAM


def cases(test):
    return next(m for m in test.pytestmark if m.name == "parametrize").args[1]


@pytest.mark.parametrize("lens,hq,hk,page,d,window", cases(T.test_attention_many_new_tokens) + cases(T.test_attention_parts))
def test_bar_of_the_kernel_that_runs(lib, lens, hq, hk, page, d, window):
    """Cases of many rows whose keys do not pay for the tensor-memory kernel, and those that do, each at its kernel's bar."""
    b = Batch(lens, hk, page, d, 120 + d + window, behind=2)
    attend(lib, b, hq, d, window, least=kernel(b, hq, hk, page, d, window))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,window", [(16, 1), (64, 1), (32, 37), (16, 100), (128, 100), (16, 300), (64, 300)])
def test_windows_on_the_tensor_memory_kernel(lib, d, page, window):
    """Windows of one key, within a key tile, across two, and across several, at every head size."""
    b = Batch([(700, 1300), (3, 40), (140, 300)], 16, page, d, 130 + d + window, behind=2)
    assert kernel(b, 32, 16, page, d, window) == TENSOR
    attend(lib, b, 32, d, window, least=TENSOR)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,window", [([(700, 1300), (140, 300)], 60), ([(200, 1300)], 0), ([(500, 900), (150, 2000)], 0)])
def test_ranges_on_the_tensor_memory_kernel(lib, d, lens, window):
    """Page scales from 0 to 1e6, whole windows of pages without a K or a V scale among them, queries of far sizes, and a
    negative scale, which turns the order of the scores."""
    b = Batch(lens, 16, 16, d, 140 + d + window)
    b.ref.scales[1][:] *= 10.0 ** b.rng.integers(-6, 7, b.ref.scales[1].shape)
    b.ref.scales[1][::3] = 0.0
    b.ref.scales[0][::4] = 0.0
    b.ref.scales[0][b.table[0, 40:50]] = 0.0
    b.ref.scales[1][b.table[0, 45:55]] = 0.0
    assert kernel(b, 32, 16, 16, d, window) == TENSOR
    attend(lib, b, 32, d, window, q_scale=8.0, least=TENSOR)
    q, _ = bf16(b.rng, b.t, 32, d)
    q = (q.float() * T.dev((10.0 ** b.rng.integers(-30, 3, (b.t, 32, 1))).astype(np.float32))).to(torch.bfloat16)
    got = lib.kv_attention(q, b.cache(lib), *b.args(), scale=-0.1, window=window)
    assert lib.get_device_error() == 0
    check_attention(got, *R.attention(q.double().cpu().numpy(), b.ref, b.table, b.start, b.kv_len, -0.1, window), least=TENSOR)


@pytest.mark.parametrize("lens,hq,hk,d,scale,window", [
    ([(150, 2700), (64, 64)], 32, 4, 128, 0.0, 0),               # the mean of the values
    ([(700, 1300), (140, 300)], 32, 16, 64, 0.0, 5),
    ([(700, 1300), (140, 300)], 32, 16, 256, 0.3, 1),            # its own value
    ([(2, 190)] * 9, 512, 4, 128, 0.1, 0),                       # three key tiles in four parts: one without any
    ([(2, 64)] * 18, 512, 4, 64, 0.1, 0),                        # one key tile in two parts
    ([(2, 190)] * 9, 512, 4, 256, 0.1, 33),
])
def test_few_and_even_keys_on_the_tensor_memory_kernel(lib, lens, hq, hk, d, scale, window):
    b = Batch(lens, hk, 16, d, 150 + d)
    assert kernel(b, hq, hk, 16, d, window) == TENSOR
    q, qx = bf16(b.rng, b.t, hq, d)
    cache, ws = b.cache(lib), lib.kv_attention_workspace(b.t, hq, hk, d, "cuda")
    out = lib.kv_attention(q, cache, *b.args(), scale=scale, window=window, workspace=ws)
    assert lib.get_device_error() == 0 and not ws[:1024].any()
    check_attention(out, *R.attention(qx, b.ref, b.table, b.start, b.kv_len, scale, window), least=TENSOR)
    ws[1024:] = 255                                              # (NaN in every partial result that is not written)
    assert torch.equal(lib.kv_attention(q, cache, *b.args(), scale=scale, window=window, workspace=ws), out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power,window", [(118, 70), (34, 300), (30, 37)])
def test_far_scores_in_windows_on_the_tensor_memory_kernel(lib, d, power, window):
    """Scores past 2^20 that first show in a tile at the window's start, and go on in tiles without a masked key."""
    lens = [(700, 1300), (140, 300)]
    assert kv_index.tensor_units(lens, 32, 16, 16, d, window)
    E.test_one_key_takes_all_the_weight(lib, d, lens, 32, 16, TENSOR, power, window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_edge_cases_reach_both_kernels(lib, d):
    assert not kv_index.tensor_units(E.FEW[0], *E.FEW[1:3], 16, d)
    assert kv_index.tensor_units(E.MANY[0], *E.MANY[1:3], 16, d)
    for page in (16, 32, 64, 128):
        assert kv_index.tensor_units([(900, 1700), (1, 333)], 32, 16, page, d, 100)
