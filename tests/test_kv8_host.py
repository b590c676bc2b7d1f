"""Checks of the 8-bit key/value cache's operators that need no GPU: argument
refusals before any launch, workspace sizes, and the plain reference against
brute force on small cases."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import kv8
from bit_weight_only_gemv_gb300 import lib

P0 = 1 << 20   # an address that is never dereferenced: every call here is refused


def structs(**over):
    c = dict(kc=P0, vc=P0, ks=P0, vs=P0, ranges=P0, weight=P0, num_pages=8, kv_heads=2,
             page_tokens=16, head_dim=64, page_stride=2048, head_stride=1024)
    b = dict(table=P0, lens=P0, offsets=None, batch=2, max_pages=4, rows=2, max_new=1, max_len=64)
    for k, v in over.items():
        (c if k in c else b)[k] = v
    return lib.KV8CacheStruct(**c), lib.KV8BatchStruct(**b)


def call(name, flags=0, k=P0, q=P0, stride=None, q_heads=4, window=0, sel=None, n_sel=None,
         max_sel=0, ws=P0, ws_bytes=1 << 30, out=P0, lse=P0, sink=0, recent=0, budget=8, kept=P0,
         new_lens=P0 + 64, dst=P0 + 128, **over):
    L = lib.load()
    c, b = structs(**over)
    cp, bp = ctypes.byref(c), ctypes.byref(b)
    st = stride if stride is not None else (128 if name == "append" else 256)
    if name == "append":
        return L.w4_kv8_append(cp, bp, k, P0, st, None, flags, None)
    if name == "attn":
        return L.w4_kv8_attn(out, lse, q, st, q_heads, cp, bp, 0.1, window, sel, n_sel, max_sel,
                             ws, ws_bytes, None, flags, None)
    if name == "select":
        return L.w4_kv8_select(sel or P0, P0, max_sel or 4, sink, recent, q, st, q_heads, cp, bp,
                               ws, ws_bytes, None, flags, None)
    if name == "weigh":
        return L.w4_kv8_weigh(q, st, q_heads, lse, cp, bp, 0.1, window, None, flags, None)
    return L.w4_kv8_evict(dst, kept, new_lens, budget, sink, recent, cp, bp, ws, ws_bytes, None,
                          flags, None)


ALL = ("append", "attn", "select", "weigh", "evict")
ARG, ALIGN, SHAPE, SPACE = 1, 2, 3, 4


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("over,code", [
    (dict(kc=None), ARG), (dict(vs=None), ARG), (dict(table=None), ARG), (dict(lens=None), ARG),
    (dict(num_pages=0), ARG), (dict(kv_heads=0), ARG), (dict(batch=0), ARG), (dict(rows=0), ARG),
    (dict(max_new=0), ARG), (dict(max_len=-1), ARG), (dict(flags=2), ARG),
    (dict(page_tokens=8), SHAPE), (dict(page_tokens=48), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(batch=5000, rows=5000), SHAPE), (dict(max_len=65), SHAPE),
    (dict(rows=3), SHAPE), (dict(max_new=2), SHAPE),          # without offsets
    (dict(kc=P0 + 8), ALIGN), (dict(page_stride=2056), ALIGN), (dict(ks=P0 + 2), ALIGN),
    (dict(lens=P0 + 2), ALIGN), (dict(ranges=P0 + 4), ALIGN),
    (dict(head_stride=512), ARG), (dict(page_stride=512), ARG),
])
def test_cache_and_batch_refusals(name, over, code):
    assert call(name, **over) == code


@pytest.mark.parametrize("name", ("attn", "select", "weigh"))
@pytest.mark.parametrize("over,code", [
    (dict(q=None), ARG), (dict(q_heads=0), ARG), (dict(q_heads=3), SHAPE),
    (dict(q_heads=2 * 129, stride=1 << 16), SHAPE), (dict(q=P0 + 8), ALIGN),
    (dict(stride=260), ALIGN), (dict(stride=248), ARG)])
def test_query_refusals(name, over, code):
    assert call(name, **over) == code


@pytest.mark.parametrize("name,over,code", [
    ("append", dict(k=None), ARG), ("append", dict(k=P0 + 2), ALIGN),
    ("append", dict(stride=120), ARG), ("append", dict(stride=132), ALIGN),
    ("attn", dict(out=None), ARG), ("attn", dict(out=P0 + 2), ALIGN), ("attn", dict(window=-1), ARG),
    ("attn", dict(lse=P0 + 2), ALIGN), ("attn", dict(sel=P0), ARG),
    ("attn", dict(sel=P0, n_sel=P0, max_sel=0), ARG),
    ("attn", dict(sel=P0, n_sel=P0, max_sel=2, offsets=P0, rows=8, max_new=4), SHAPE),
    ("select", dict(ranges=None), ARG), ("select", dict(sink=3, recent=2), ARG),
    ("select", dict(ws=None), SPACE), ("select", dict(ws_bytes=16), SPACE),
    ("select", dict(ws=P0 + 8), ALIGN), ("select", dict(offsets=P0, rows=8, max_new=4), SHAPE),
    ("weigh", dict(weight=None), ARG), ("weigh", dict(lse=None), ARG),
    ("weigh", dict(window=-2), ARG),
    ("evict", dict(weight=None), ARG), ("evict", dict(budget=0), ARG),
    ("evict", dict(sink=5, recent=4), ARG), ("evict", dict(ws_bytes=16), SPACE),
    ("evict", dict(new_lens=P0), ARG), ("evict", dict(dst=P0), ARG), ("evict", dict(kept=None), ARG),
])
def test_call_refusals(name, over, code):
    assert call(name, **over) == code


def test_workspace_sizes():
    L = lib.load()
    c, b = structs()
    bad, _ = structs(head_dim=96)
    assert L.w4_kv8_select_workspace_bytes(ctypes.byref(c), ctypes.byref(b)) >= 2 * 2 * (4 + 4 * 4)
    assert L.w4_kv8_select_workspace_bytes(ctypes.byref(bad), ctypes.byref(b)) == 0
    assert L.w4_kv8_evict_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8) >= 2 * 2 * 64 * 4
    assert L.w4_kv8_evict_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 0) == 0
    assert L.w4_kv8_attn_workspace_bytes(ctypes.byref(bad), ctypes.byref(b), 4, 0) == 0


# ------------------------------------------------------------------ the reference's own pins
def test_least_step_is_the_least():
    for m in (0.0, 1e-40, 2.0 ** -94, 127.0, 127.5, 1.0, 1.9921875, 3.3e38, 254 / 256, 0.9921875):
        s = kv8.least_step(m)
        assert s >= 2.0 ** -100 and Fraction(m) <= 127 * Fraction(s)
        assert s == 2.0 ** -100 or Fraction(m) > 127 * Fraction(s) / 2


def test_top_takes_ties_from_the_lowest_index():
    assert kv8.top([1, 3, 3, 0, 3], 2) == [1, 2]
    assert kv8.top([2.0, 2.0, 2.0], 3) == [0, 1, 2]


def test_attention_reference_by_hand():
    """Two keys, one head: weights e^0 and e^1 over their sum."""
    kc = np.full((1, 1, 16, 64), 128, np.uint8)
    kc[0, 0, 1, 0] = 129
    vc = np.full((1, 1, 16, 64), 128, np.uint8)
    vc[0, 0, 0], vc[0, 0, 1] = 130, 132
    one = np.ones((1, 1), np.float32)
    cache = {"kc": kc, "vc": vc, "ks": one, "vs": one}
    q = np.zeros((1, 1, 64))
    q[0, 0, 0] = 1.0
    out, lse, _, _ = kv8.attn_ref(cache, np.zeros((1, 1), np.int32), [2], None, q, 1.0)
    e = np.e
    assert np.allclose(out[0, 0], (2 + 4 * e) / (1 + e)) and np.allclose(lse, np.log(1 + e))
    out, lse, _, _ = kv8.attn_ref(cache, np.zeros((1, 1), np.int32), [2], None, q, 1.0, window=1)
    assert np.all(out == 4) and np.allclose(lse, 1)


def test_weigh_reference_adds_one_per_row_and_head():
    rng = np.random.default_rng(0)
    cache = {"kc": rng.integers(0, 256, (3, 1, 16, 64)).astype(np.uint8),
             "vc": rng.integers(0, 256, (3, 1, 16, 64)).astype(np.uint8),
             "ks": np.full((3, 1), 0.01, np.float32), "vs": np.full((3, 1), 0.01, np.float32),
             "weight": np.zeros((3, 1, 16), np.float32)}
    table, q = np.array([[2, 0, 1]], np.int32), rng.normal(size=(5, 3, 64))
    _, lse, _, _ = kv8.attn_ref(cache, table, [40], [0, 5], q, 0.1)
    w, _ = kv8.weigh_ref(cache, table, [40], [0, 5], q, lse, 0.1)
    assert np.isclose(w.sum(), 15) and np.all(w[1, 0, 8:] == 0)


def test_python_checks():
    t = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.KV8Batch(t, torch.zeros(2, dtype=torch.int32), max_len=8)         # not on the GPU
    with pytest.raises(ValueError):
        lib.KV8Cache(torch.zeros((1, 1, 16, 64), dtype=torch.uint8),
                     torch.zeros((1, 1, 16, 64), dtype=torch.uint8),
                     torch.zeros((1, 1)), torch.zeros((1, 1)))
