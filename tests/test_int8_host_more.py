"""Host-side checks of the 8-bit integer path that need no GPU, beside those of test_int8_host.py."""

import ctypes

import pytest

from test_int8_host import SHAPE, B, P, _attend, _heads, _qk, _update, lib  # noqa: F401  (fixtures)


@pytest.mark.parametrize("strides", [dict(token=1024), dict(token=128, head=384), dict(head=256, token=1024)])
def test_an_output_that_is_its_input_has_its_strides(B, lib, strides):  # noqa: F811
    """Three tokens of four heads of 128: written in place under other strides, rows would be overwritten unread."""
    other = _heads(B, **strides)
    assert _qk(B, lib, qo=other) == SHAPE
    assert _qk(B, lib, q=other) == SHAPE
    assert lib.w4a8_qk_norm_rope(None, ctypes.byref(_heads(B)), 3, 128, None, None, 1e-6, None, None, None,
                                 ctypes.byref(other), None) == SHAPE
    assert _update(B, lib, q=_heads(B), qo=other) == SHAPE
    assert _attend(B, lib, out=other) == SHAPE
