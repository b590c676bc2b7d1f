"""Corners of the 8-bit cache's contract: special weights, pages that are none, steps at the ends
of their range, light tokens beside heavy ones."""

import numpy as np
import pytest
import torch

from oracle import kv8
from bit_weight_only_gemv_gb300 import lib
from _kv8 import Case, bf16_round, check_attn, score_error

pytestmark = pytest.mark.gpu

ERR = lib.STATUS_CODE["W4_ERR_INDEX"]


def status(c):
    torch.cuda.synchronize()
    return int(c.status.item())


@pytest.mark.parametrize("n", [32, 9000, 17000])
def test_evict_takes_any_nan_as_the_largest(cuda_lib, n):
    """NaNs of either sign and any payload are equal to one another: the lowest positions first."""
    c = Case(193, [n], None, 1, 64, 16, spare=1)
    w = np.full(n, 2.0, np.float32)
    w[15] = np.inf
    bits = w.view(np.uint32)
    bits[3], bits[7], bits[11], bits[20] = 0xFFC00000, 0x7FFFFFFF, 0xFF800001, 0x7F800001
    pages = -(-n // 16)
    c.cache["weight"][c.table[0, :pages], 0] = np.resize(w, (pages, 16))
    c.to_gpu()
    for budget, want in ((2, [3, 7]), (4, [3, 7, 11, 20]), (6, [0, 3, 7, 11, 15, 20])):
        ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, budget))
        kept, _ = lib.kv8_evict(c.dev, c.batch, budget,
                                torch.from_numpy(c.free[:1][None].copy()).cuda(), 0, 0, ws, c.status)
        assert status(c) == 0
        assert kept.flatten().tolist() == want


# log2 of the levels' weights against the heaviest, and the order in which the levels come: the
# second of each pair rises above what came first by less than what moves a running maximum, the
# third by more than fp32's range of exponents
LEVELS = (0, -25, -60, -90, -118)
ORDERS = {"rising": (4, 3, 2, 1, 0), "falling": (0, 1, 2, 3, 4), "lagging": ("far", 3, 0, 4, 1),
          "lagging twice": ("far", 4, 2, 0, 3), "scattered": None}


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("length", [200, 3000])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [None, 20, 70])
def test_attn_light_tokens_keep_their_bits(cuda_lib, new, D, length, order):
    """Tokens of five levels of weight, each alone in channels of its own (the others hold code
    128, zero there): every level shows at its own size, however light."""
    c = Case(3, [length], None if new is None else [new], 1, D, 32, 8)
    levels = ORDERS[order]
    pos = np.arange(length)
    if levels is None:
        level = c.rng.integers(0, 5, length)
        x = np.array(LEVELS)[level]
    else:
        part = pos * 5 // length
        level = np.array([4 if p == "far" else p for p in levels])[part]
        # "far": 55 below the next level and further below the heaviest than 2^-126
        x = np.array([LEVELS[levels[1]] - 55 if p == "far" else LEVELS[p] for p in levels])[part]
    c.cache["kc"][:], c.cache["vc"][:] = 128, 128
    c.cache["ks"][:], c.cache["vs"][:] = 1.0, 0.25
    page, slot = c.table[0, pos // 32], pos % 32
    c.cache["kc"][page, 0, slot, 0] = 228 + x
    for g in range(5):
        t = np.flatnonzero(level == g)
        ch = np.arange(g, D, 5)
        c.cache["vc"][page[t][:, None], 0, slot[t][:, None], ch] = \
            c.rng.integers(129, 256, (len(t), len(ch)))
    c.q[:] = 0
    c.q[:, :, 0] = 1
    c.scale = float(np.log(2.0))      # a score is the code, in powers of two
    c.to_gpu()
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    assert ref[0][-1].max() > 1 and 0 < ref[0][ref[0] > 0].min() < 2.0 ** -80
    out, lse = c.attn()
    assert status(c) == 0
    check_attn(out, lse, ref, D)
