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
