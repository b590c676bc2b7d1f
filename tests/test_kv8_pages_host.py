"""Refusals of w4_kv8_weigh_pages that need no GPU."""

import ctypes

import pytest

from bit_weight_only_gemv_gb300 import lib
from test_kv8_host import ALIGN, ARG, P0, SHAPE, structs


@pytest.mark.parametrize("sel,n_sel,max_sel,over,code", [
    (P0, None, 2, {}, ARG), (None, P0, 2, {}, ARG), (P0, P0, 0, {}, ARG), (P0, P0, -1, {}, ARG),
    (P0 + 2, P0, 2, {}, ALIGN), (P0, P0 + 2, 2, {}, ALIGN), (P0, P0, (1 << 24) + 1, {}, SHAPE),
    (P0, P0, 2, dict(offsets=P0, rows=8, max_new=4), SHAPE),
    (P0, P0, 2, dict(weight=None), ARG), (P0, P0, 2, dict(head_dim=96), SHAPE),
])
def test_refusals(sel, n_sel, max_sel, over, code):
    c, b = structs(**over)
    assert lib.load().w4_kv8_weigh_pages(P0, 256, 4, P0, ctypes.byref(c), ctypes.byref(b), 0.1, 0,
                                         sel, n_sel, max_sel, None, 0, None) == code


@pytest.mark.parametrize("q,stride,heads,lse,window,flags,code", [
    (None, 256, 4, P0, 0, 0, ARG), (P0, 256, 3, P0, 0, 0, SHAPE), (P0, 260, 4, P0, 0, 0, ALIGN),
    (P0, 248, 4, P0, 0, 0, ARG), (P0, 256, 4, None, 0, 0, ARG), (P0, 256, 4, P0 + 2, 0, 0, ALIGN),
    (P0, 256, 4, P0, -1, 0, ARG), (P0, 256, 4, P0, 0, 2, ARG)])
def test_query_refusals(q, stride, heads, lse, window, flags, code):
    c, b = structs()
    assert lib.load().w4_kv8_weigh_pages(q, stride, heads, lse, ctypes.byref(c), ctypes.byref(b), 0.1,
                                         window, P0, P0, 2, None, flags, None) == code
