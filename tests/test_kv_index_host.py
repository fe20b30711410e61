"""The int8 paged cache's index arithmetic (csrc/kv_index.h), compiled for the host."""

import numpy as np
import pytest

import kv_index


def test_pages_that_a_range_sees():
    """A group of 16 keys before a range's end is looked up exactly if its page has a key of the range."""
    f = kv_index.library().first_key
    for shift in (4, 5, 6, 7):
        page = 1 << shift
        for lo, hi in ((0, 1), (0, 300), (17, 18), (100, 300), (127, 129), (128, 400), (255, 256)):
            for key in range(0, hi, 16):
                keys = range(key // page * page, (key // page + 1) * page)
                assert (key >= f(lo, hi, shift)) == any(k >= lo for k in keys), (lo, hi, key, shift)
    assert f(2 ** 30 - 1, 2 ** 30, 7) == 2 ** 30 - 128


@pytest.mark.parametrize("ctas", [148, 160, 132])
def test_every_item_has_one_cta_of_the_kernels(ctas):
    """The streaming kernel's split of its items: contiguous shares that cover every item once, none empty, and the CTA
    named for an item holds it."""
    lib = kv_index.library()
    for total in (1, 2, 3, 7, 147, 148, 149, 1000, 4097, 2 ** 40 + 12345):
        n = min(total, ctas)
        edges = [lib.first_item(c, total, n) for c in range(n + 1)]
        assert edges[0] == 0 and edges[-1] == total and all(a < b for a, b in zip(edges, edges[1:]))
        for i in range(total) if total < 10 ** 5 else [e + o for e in edges[:-1] for o in (0, 1)] + [e - 1 for e in edges[1:]]:
            c = lib.item_cta(i, total, n)
            assert edges[c] <= i < edges[c + 1]


def test_tiles_stay_within_the_launch():
    """The host's bound on the row tiles, which sizes the launch, holds for any split of the rows into sequences."""
    lib, rng = kv_index.library(), np.random.default_rng(1)
    for _ in range(500):
        group, tile = int(rng.integers(1, 129)), int(rng.choice([128, 256]))
        lens = rng.integers(0, 400, int(rng.integers(1, 9)))
        tiles = sum(-(-int(n) * group // tile) for n in lens if n * group >= 128)
        assert tiles <= lib.tiles_bound(int(lens.sum()) * group, len(lens), tile)


def test_no_tiles_without_rows():
    """Decode steps, and sequences below 128 rows, are the streaming kernel's whatever their keys."""
    assert kv_index.tensor_units([(1, 10 ** 6)] * 64, 32, 8, 64, 128) == 0
    assert kv_index.tensor_units([(31, 10 ** 6)] * 64, 32, 8, 64, 128) == 0
    assert kv_index.tensor_units([(32, 10 ** 6)] * 64, 32, 8, 64, 128) == 64 * 8
    assert kv_index.tensor_units([(2048, 8192)] * 2, 32, 8, 64, 128) == 2 * 8192 // 256 * 8
