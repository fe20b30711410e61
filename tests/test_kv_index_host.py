"""The int8 paged cache's index arithmetic (csrc/kv_index.h), compiled for the host."""

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
