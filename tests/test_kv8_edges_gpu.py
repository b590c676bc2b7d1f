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


def good_or_unwritten(c, out, lse, ref, blind):
    """Rows `blind` (bool [rows]) unwritten, every other one right, or unwritten in all channels of
    one head."""
    assert np.isnan(out[blind]).all() and np.isnan(lse[blind]).all()
    left = np.isnan(lse)
    assert np.array_equal(left, np.isnan(out).all(-1)) and np.array_equal(left, np.isnan(out).any(-1))
    rows, heads = np.nonzero(~left)
    check_attn(out[rows, heads], lse[rows, heads], [x[rows, heads] for x in ref], c.D)
    return left


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [3, 100])
def test_attn_rows_that_see_a_bad_page_stay_unwritten(cuda_lib, new, D, long):
    """A page that is none among the new tokens' own: rows before it do not see it.  Few rows (the
    token kernel) and many (several row tiles of the chunk kernel), units whole and cut."""
    length = (5000 if long else 300) + new
    c = Case(7 * D + new, [150, length, 90], [2, new, 2], 2, D, 16, 8)
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    first = length - new
    pos = np.full(c.rows, -1)
    pos[2:2 + new] = first + np.arange(new)
    for page in (0, (first + new * 3 // 5) // 16, (length - 1) // 16):
        keep = c.table[1, page]
        c.table[1, page] = c.cache["ks"].shape[0] if page else -3
        c.to_gpu()
        blind = pos >= page * 16
        left = good_or_unwritten(c, *c.attn(), ref, blind)
        assert status(c) == ERR
        assert not left[:2].any() and not left[2 + new:].any()   # other sequences
        if new == 100 and 16 < page < (length - 1) // 16:        # row tiles before the page
            assert not left[2:2 + 16].any()
        c.table[1, page] = keep
    c.to_gpu()
    c.batch.tensors[1][1] = length + 1                           # a length past the bound
    left = good_or_unwritten(c, *c.attn(), ref, pos >= 0)
    assert status(c) == ERR
    assert not left[:2].any() and not left[2 + new:].any()


@pytest.mark.parametrize("D", [64, 256])
def test_attn_refusals_among_thousands_of_units(cuda_lib, D):
    """Many units a CTA, a third of them with a page that is none: the others' bits as without."""
    B = 700
    rng = np.random.default_rng(D)
    c = Case(D, [int(x) for x in rng.integers(1, 50, B)], None, 8, D, 16, 128)
    c.to_gpu()
    out, lse = c.attn()
    assert status(c) == 0 and not np.isnan(out).any()
    bad = rng.random(B) < 0.33
    for b in np.flatnonzero(bad):
        c.table[b, rng.integers(0, -(-c.lens[b] // 16))] = 1 << 30
    c.to_gpu()
    out2, lse2 = c.attn()
    assert status(c) == ERR
    assert np.isnan(out2[bad]).all() and np.isnan(lse2[bad]).all()
    assert np.array_equal(out[~bad], out2[~bad]) and np.array_equal(lse[~bad], lse2[~bad])


def test_append_stores_all_but_a_bad_page(cuda_lib):
    c = Case(8, [100, 70], [80, 30], 2, 64, 16)
    c.fix_ranges([20, 40])
    k, v = (bf16_round(c.rng.normal(size=(c.rows, 2, 64))) for _ in range(2))
    want = kv8.append_ref(c.cache, c.table, c.lens, c.offsets, k, v)
    page = c.table[0, 3]
    for n in want:
        want[n][page] = c.cache[n][page]
    c.table[0, 3] = -1
    c.to_gpu()
    lib.kv8_append(c.dev, c.batch, *(torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (k, v)),
                   c.status)
    assert status(c) == ERR
    got = c.dev_arrays()
    assert all(np.array_equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("vstep", [0.0, 2.0 ** -100, 2.0 ** -6 * 1.3, 2.0 ** 30])
@pytest.mark.parametrize("rise", [0, 59, 110])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [None, 30])
def test_attn_steps_at_the_ends_of_their_range(cuda_lib, new, D, rise, vstep):
    """Thousands of tokens 2^rise above the first ones, in values of every allowed size: below
    what moves the chunk kernel's maximum, and above."""
    n = 2500
    c = Case(17, [n], None if new is None else [new], 1, D, 64, 8)
    c.cache["kc"][:] = 128
    c.cache["ks"][:] = 2.0 ** 30
    c.cache["vs"][:] = vstep
    pos = np.arange(n)
    c.cache["kc"][c.table[0, pos // 64], 0, pos % 64, 0] = np.where(pos < 40, 128, 128 + rise)
    c.q[:] = 0
    c.q[:, :, 0] = 2.0 ** -30
    c.scale = float(np.log(2.0))
    c.to_gpu()
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    out, lse = c.attn()
    assert status(c) == 0
    check_attn(out, lse, ref, D)


def moved(c, layout):
    """The case's cache with its pages and heads elsewhere: gaps that no head's size divides, or
    all pages of a head side by side."""
    n, H, P, D = c.cache["kc"].shape
    out = []
    for name in ("kc", "vc"):
        if layout == "gaps":
            strides = (H * (P * D + 16) + 48, P * D + 16, D, 1)
            size = strides[0] * n
        else:
            strides = (P * D, n * P * D + 32, D, 1)
            size = strides[1] * H
        t = torch.as_strided(torch.full((size,), 77, dtype=torch.uint8, device="cuda"),
                             (n, H, P, D), strides)
        t.copy_(torch.from_numpy(c.cache[name]))
        out.append(t)
    rest = c.dev.tensors
    c.dev = lib.KV8Cache(*out, rest[2], rest[3], ranges=rest[4], weight=rest[5])


@pytest.mark.parametrize("layout", ["gaps", "heads first"])
@pytest.mark.parametrize("D,P,news", [(64, 16, None), (128, 32, [1, 40]), (256, 128, [30, 9]),
                                      (64, 64, [70, 3]), (128, 16, None)])
def test_pages_and_heads_anywhere(cuda_lib, D, P, news, layout):
    """Every operator on strides other than the dense ones."""
    c = Case(5 + D, [150, 333], news, 3, D, P, 4, spare=8)
    before = [150, 333] if news is None else [150 - news[0], 333 - news[1]]
    c.fix_ranges([n - (news is None) for n in before])
    k, v = (bf16_round(c.rng.normal(size=(c.rows, 3, D))) for _ in range(2))
    c.to_gpu()
    moved(c, layout)
    want = kv8.append_ref(c.cache, c.table, c.lens, c.offsets, k, v)
    lib.kv8_append(c.dev, c.batch, *(torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (k, v)),
                   c.status)
    assert status(c) == 0
    got = c.dev_arrays()
    assert all(np.array_equal(got[n], want[n]) for n in want)
    c.cache = want
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    out, lse = c.attn()
    assert status(c) == 0
    check_attn(out, lse, ref, D)
    lse = ref[1].astype(np.float32)
    after, reach = kv8.weigh_ref(c.cache, c.table, c.lens, c.offsets, c.q, lse.astype(np.float64),
                                 c.scale)
    lib.kv8_weigh(c.dev, c.batch, c.gpu_q(), torch.from_numpy(lse).cuda(), c.scale, 0, c.status)
    assert status(c) == 0
    weight = c.dev_arrays()["weight"]
    added = after - c.cache["weight"]
    assert np.all(np.abs(weight - after) <= score_error(D, reach) + 2.0 ** -20 * added +
                  2.0 ** -22 * after + c.max_new * 4 * 2.0 ** -24 * added)
    c.cache["weight"] = weight
    if news is None:
        ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
        sel, n_sel = lib.kv8_select(c.dev, c.batch, c.gpu_q(), 5, 1, 1, ws, c.status)
        want_sel, want_n = kv8.select_ref(c.cache, c.table, c.lens, c.q, 5, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want_sel)
        out, lse = c.attn(sel=sel, n_sel=n_sel)
        assert status(c) == 0
        check_attn(out, lse, kv8.attn_ref(c.cache, c.table, c.lens, None, c.q, c.scale, 0, want_sel,
                                          want_n), D)
    pages = -(-48 // P)
    dst = c.free[:2 * pages].reshape(2, pages).copy()
    want, kept, _ = kv8.evict_ref(c.cache, c.table, c.lens, dst, 48, 2, 8)
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, 48))
    got_kept, _ = lib.kv8_evict(c.dev, c.batch, 48, torch.from_numpy(dst).cuda(), 2, 8, ws, c.status)
    assert status(c) == 0 and np.array_equal(got_kept.cpu().numpy(), kept)
    got = c.dev_arrays()
    assert all(np.array_equal(got[n], want[n]) for n in want)
