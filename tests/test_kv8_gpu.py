"""GPU parity of the 8-bit key/value cache's operators against the plain fp64
reference, at the sizes and masks where they can go wrong."""

import numpy as np
import pytest
import torch

from oracle import kv8
from bit_weight_only_gemv_gb300 import lib
from _kv8 import Case, bf16_round, check_attn, score_error

pytestmark = pytest.mark.gpu


def status(c):
    torch.cuda.synchronize()
    return int(c.status.item())


def same(got, want):
    for n in want:
        assert np.array_equal(got[n], want[n]), (n, np.argwhere(got[n] != want[n])[:5])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("lens,news,H,D,P,layered", [
    ([1], None, 1, 64, 16, False),                              # the first token of all
    ([5, 17, 33, 48], None, 2, 128, 16, False),                 # inside, first and last of a page
    ([40, 1, 64, 129], [40, 1, 3, 65], 3, 128, 32, True),       # whole prompts and tails
    ([300, 77], [256, 0], 2, 256, 64, False),                   # no new row for the second
    ([200], [130], 1, 64, 128, False),
    ([0, 9], None, 2, 64, 16, False),                           # a padded slot of the batch
])
def test_append(cuda_lib, lens, news, H, D, P, layered):
    c = Case(len(lens) * 7 + D, lens, news, H, D, P)
    before = [n - (1 if news is None else news[i]) for i, n in enumerate(lens)]
    c.fix_ranges([max(0, n) for n in before])
    size = np.exp(c.rng.normal(size=(c.rows, H, 1)) * 2)
    k, v = (bf16_round(c.rng.normal(size=(c.rows, H, D)) * size) for _ in range(2))
    k[0, 0], v[-1, -1] = 0.0, 0.0                               # a block of zeros alone
    c.to_gpu(layered=layered)
    qkv = torch.zeros((c.rows, 3 * H, D), dtype=torch.bfloat16, device="cuda")
    qkv[:, H:2 * H] = torch.from_numpy(k).cuda().to(torch.bfloat16)
    qkv[:, 2 * H:] = torch.from_numpy(v).cuda().to(torch.bfloat16)
    want = kv8.append_ref(c.cache, c.table, c.lens, c.offsets, k, v)
    for _ in range(2):                                          # the second call changes nothing
        lib.kv8_append(c.dev, c.batch, qkv[:, H:2 * H], qkv[:, 2 * H:], c.status)
        assert status(c) == 0
        same(c.dev_arrays(), want)


def test_append_token_by_token_equals_one_call_of_equal_steps(cuda_lib):
    """Values whose largest comes first: no step grows later, so order does not matter."""
    c = Case(3, [40], [40], 2, 64, 16)
    x = bf16_round(c.rng.normal(size=(40, 2, 64)).clip(-3, 3))
    x[::16, :, 0] = 3.5
    c.to_gpu()
    t = torch.from_numpy(x).cuda().to(torch.bfloat16)
    lib.kv8_append(c.dev, c.batch, t, t, c.status)
    one = c.dev_arrays()
    d = Case(3, [40], None, 2, 64, 16)
    d.cache = {n: a.copy() for n, a in c.cache.items()}
    d.to_gpu()
    for i in range(40):
        d.batch.tensors[1].fill_(i + 1)
        lib.kv8_append(d.dev, d.batch, t[i:i + 1], t[i:i + 1], d.status)
    assert status(c) == 0 and status(d) == 0
    same(d.dev_arrays(), one)


def test_append_round_trip_error(cuda_lib):
    """A stored value is within half a step of its input, a step at most m / 63.5."""
    c = Case(5, [96], [96], 1, 128, 32)
    x = bf16_round(c.rng.normal(size=(96, 1, 128)) * np.exp(c.rng.normal(size=(96, 1, 1))))
    c.to_gpu()
    t = torch.from_numpy(x).cuda().to(torch.bfloat16)
    lib.kv8_append(c.dev, c.batch, t, t, c.status)
    a = c.dev_arrays()
    for i in range(3):
        pg, part = c.table[0, i], x[32 * i:32 * i + 32, 0]
        for codes, steps in ((a["kc"], a["ks"]), (a["vc"], a["vs"])):
            step = float(steps[pg, 0])
            assert np.abs(part).max() / 127 <= step < 2 * np.abs(part).max() / 127
            assert np.all(np.abs((codes[pg, 0].astype(float) - 128) * step - part) <= step / 2)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_append_refuses_values_that_are_not_finite(cuda_lib, value):
    c = Case(9, [20, 20], None, 2, 64, 16)
    c.fix_ranges([19, 19])
    k, v = (bf16_round(c.rng.normal(size=(2, 2, 64))) for _ in range(2))
    want = kv8.append_ref(c.cache, c.table, c.lens, None, k, v)
    pg = c.table[1, 1]
    for n in ("kc", "ks", "ranges"):
        want[n][pg, 0] = c.cache[n][pg, 0]
    c.to_gpu()
    kt, vt = (torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (k, v))
    kt[1, 0, 37] = value
    lib.kv8_append(c.dev, c.batch, kt, vt, c.status)
    assert status(c) == lib.STATUS_CODE["W4_ERR_VALUE"]
    same(c.dev_arrays(), want)


# ------------------------------------------------------------------ attention
ATTN = [
    # lens, news, H, D, P, G, window
    ([1], None, 1, 64, 16, 1, 0),
    ([1, 15, 16, 17, 200], None, 2, 128, 16, 4, 0),
    ([0, 3, 0], None, 1, 128, 32, 8, 0),                  # empty sequences of a padded batch
    ([700], None, 2, 256, 16, 4, 512),
    ([513, 64, 1000], None, 1, 64, 128, 16, 100),
    ([333], None, 2, 128, 64, 3, 1),                      # a window of one: the token itself
    ([2000], None, 1, 128, 32, 71, 0),                    # an odd group wider than one tile
    ([50, 40], [3, 2], 2, 64, 16, 5, 0),
    ([130], [130], 1, 128, 32, 2, 0),                     # a whole prompt
    ([300, 7, 0, 129], [100, 7, 0, 1], 2, 64, 16, 3, 0),
    ([1000, 260], [256, 33], 1, 128, 64, 4, 200),
    ([400], [250], 1, 256, 32, 2, 0),
    ([90], [64], 3, 256, 16, 6, 10),
    ([5000], [17], 1, 128, 128, 8, 0),
    ([3], [9], 1, 64, 16, 2, 0),                          # rows at negative positions
]


@pytest.mark.parametrize("lens,news,H,D,P,G,window", ATTN)
@pytest.mark.parametrize("pow2", [True, False])
def test_attn(cuda_lib, lens, news, H, D, P, G, window, pow2):
    c = Case(sum(lens) + D + G, lens, news, H, D, P, G, pow2=pow2)
    c.to_gpu(layered=pow2)
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale, window)
    out, lse = c.attn(window)
    assert status(c) == 0
    check_attn(out, lse, ref, D)
    again = c.attn(window)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("news", [None, [3, 70]])
def test_attn_does_not_read_what_is_masked(cuda_lib, news):
    """Pages past the lengths, steps of other pages, codes past the length: never in a sum."""
    c = Case(21, [100, 150], news, 2, 128, 32, 4)
    used = set(c.table[c.table >= 0].tolist())
    for pg in range(c.cache["ks"].shape[0]):
        if pg not in used:
            c.cache["ks"][pg], c.cache["vs"][pg] = np.nan, np.inf
    c.to_gpu()
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    out, lse = c.attn()
    check_attn(out, lse, ref, 128)
    for b, n in enumerate(c.lens):                        # other codes in the last pages' tails
        pg = c.table[b, (n - 1) // 32]
        c.cache["kc"][pg, :, n % 32:], c.cache["vc"][pg, :, n % 32:] = 255, 0
    c.to_gpu()
    again = c.attn()
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("news", [None, [40, 30]])
def test_attn_nan_query_rows_stay_alone(cuda_lib, news):
    c = Case(22, [100, 50], news, 1, 64, 16, 4)
    c.to_gpu()
    out, lse = c.attn()
    q = c.gpu_q()
    q[1, 2, 5] = float("nan")
    out2, lse2 = c.attn(q=q)
    assert np.isnan(out2[1, 2]).all() and np.isnan(lse2[1, 2])
    out2[1, 2], lse2[1, 2] = out[1, 2], lse[1, 2]
    assert np.array_equal(out, out2) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("news", [None, [33]])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 1e3, 1e30])
def test_attn_extreme_queries_and_steps(cuda_lib, size, news):
    """Queries of any size, value steps spread over 2^-60 .. 2^20, scores of hundreds."""
    c = Case(23, [400], news, 1, 128, 16, 8, pow2=False)
    c.cache["vs"] = (2.0 ** c.rng.integers(-60, 20, c.cache["vs"].shape)).astype(np.float32)
    c.q = bf16_round(c.q * size)
    c.scale = 128 ** -0.5 / size * 4
    c.to_gpu()
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    out, lse = c.attn()
    # a value step 2^-s of the largest in use leaves an absolute error of its
    # own: p rounded to a multiple of 2^-30 of the row's largest, times 127
    big = 127 * c.cache["vs"][c.table[0]].max()
    keep = ref[2].copy()
    keep += big * 2.0 ** -16
    check_attn(out, lse, (ref[0], ref[1], keep, ref[3]), 128)


def test_attn_zero_steps(cuda_lib):
    c = Case(24, [70], None, 1, 64, 16, 2)
    c.cache["vs"][:] = 0
    c.cache["ks"][:] = 0
    c.to_gpu()
    out, lse = c.attn()
    assert np.all(out == 0)
    assert np.all(np.abs(lse - np.log(70)) < 1e-5)


def test_attn_sequence_bounds_and_bad_pages_leave_rows_unwritten(cuda_lib):
    err = lib.STATUS_CODE["W4_ERR_INDEX"]
    for news in (None, [2, 40, 2]):
        c = Case(25, [100, 90, 80], news, 2, 64, 16, 2)
        c.table[1, 2] = 10 ** 6
        c.to_gpu()
        rows = slice(1, 2) if news is None else slice(2, 42)
        good = np.ones(c.rows, bool)
        good[rows] = False
        out, lse = c.attn()
        assert status(c) == err
        assert np.isnan(out[rows]).all() and np.isnan(lse[rows]).all()
        c.table[1, 2] = c.table[0, 0]
        ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
        check_attn(out[good], lse[good], [x[good] for x in ref], 64)
        # a length past the bound
        d = Case(25, [100, 90, 80], news, 2, 64, 16, 2)
        d.to_gpu()
        d.batch.tensors[1][1] = 101
        out, lse = d.attn()
        assert status(d) == err
        assert np.isnan(out[rows]).all()
        check_attn(out[good], lse[good], [x[good] for x in ref], 64)


def test_attn_strided_queries_other_stream_and_graph(cuda_lib):
    c = Case(26, [300, 200], None, 2, 128, 32, 4)
    c.to_gpu()
    want = c.attn()
    wide = torch.zeros((2, 16, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 4:12] = c.gpu_q()
    got = c.attn(q=wide[:, 4:12])
    assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])
    out = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    q = c.gpu_q()
    ws = c.scratch(lib.kv8_attn_workspace_bytes(c.dev, c.batch, 8))
    call = lib.bind_kv8_attn(c.dev, c.batch, q, c.scale, out, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0])
    with torch.cuda.graph(graph, stream=side):
        call()
        call(pdl=True)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0])


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("lens,H,D,P,G,max_sel,sink,recent", [
    ([1], 1, 64, 16, 1, 1, 0, 0),
    ([500, 3, 160, 0], 2, 128, 16, 4, 8, 1, 2),
    ([5000], 1, 256, 16, 8, 40, 0, 0),
    ([1000, 2000], 3, 64, 32, 3, 100, 2, 1),
    ([33000], 1, 128, 16, 2, 64, 1, 1),                   # more pages than one CTA scores at once
])
def test_select_and_sparse_attention(cuda_lib, lens, H, D, P, G, max_sel, sink, recent):
    c = Case(sum(lens) + P, lens, None, H, D, P, G)
    c.fix_ranges()
    c.to_gpu()
    ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
    want, n_want = kv8.select_ref(c.cache, c.table, c.lens, c.q, max_sel, sink, recent)
    for _ in range(2):
        sel, n_sel = lib.kv8_select(c.dev, c.batch, c.gpu_q(), max_sel, sink, recent, ws, c.status)
        assert status(c) == 0
        assert np.array_equal(n_sel.cpu().numpy(), n_want)
        assert np.array_equal(sel.cpu().numpy(), want)
    out, lse = c.attn(sel=sel, n_sel=n_sel)
    assert status(c) == 0
    ref = kv8.attn_ref(c.cache, c.table, c.lens, None, c.q, c.scale, 0, want, n_want)
    check_attn(out, lse, ref, D)


def test_select_ties_take_the_lowest_pages(cuda_lib):
    c = Case(31, [64 * 16], None, 1, 64, 16, 2)
    c.cache["kc"][:], c.cache["ks"][:] = 200, 0.5
    c.fix_ranges()
    c.to_gpu()
    ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
    sel, _ = lib.kv8_select(c.dev, c.batch, c.gpu_q(), 7, 0, 2, ws, c.status)
    assert sel.flatten().tolist() == [0, 1, 2, 3, 4, 62, 63]


def test_score_is_an_upper_bound_of_the_best_key(cuda_lib):
    """With the query's rounding allowed for, no key of an unchosen page has a group sum above
    the page's score."""
    c = Case(32, [640], None, 1, 128, 16, 4)
    c.fix_ranges()
    x = c.q[0]
    up, down = np.maximum(x, 0).sum(0), np.minimum(x, 0).sum(0)
    u = kv8.least_step(max(up.max(), -down.min()))
    for i in range(40):
        pg = c.table[0, i]
        lo, hi = c.cache["ranges"][pg, 0].astype(float) - 128
        score = float(hi @ np.rint(up / u) + lo @ np.rint(down / u)) * float(c.cache["ks"][pg, 0]) * u
        keys = (c.cache["kc"][pg, 0].astype(float) - 128) * float(c.cache["ks"][pg, 0])
        slack = u / 2 * (np.abs(hi) + np.abs(lo)).sum() * float(c.cache["ks"][pg, 0])
        assert (keys @ x.sum(0)).max() <= score + slack


def test_sparse_attention_bad_and_empty_selections(cuda_lib):
    c = Case(33, [100, 90, 80], None, 1, 64, 16, 2)
    c.to_gpu()
    sel = torch.tensor([[[0, 3, 6, -1]], [[1, 2, 9, -1]], [[0, 0, 0, 0]]], dtype=torch.int32,
                       device="cuda")
    n_sel = torch.tensor([[3], [3], [0]], dtype=torch.int32, device="cuda")
    out, lse = c.attn(sel=sel, n_sel=n_sel)
    assert status(c) == lib.STATUS_CODE["W4_ERR_INDEX"]
    assert np.isnan(out[1]).all() and np.all(out[2] == 0) and np.all(np.isneginf(lse[2]))
    ref = kv8.attn_ref(c.cache, c.table, c.lens, None, c.q, c.scale, 0, sel.cpu().numpy(),
                       n_sel.cpu().numpy())
    check_attn(out[[0]], lse[[0]], [x[[0]] for x in ref], 64)


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("lens,news,H,D,P,G,window", ATTN)
def test_weigh(cuda_lib, lens, news, H, D, P, G, window):
    c = Case(sum(lens) + D, lens, news, H, D, P, G)
    c.to_gpu()
    _, lse, _, _ = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale, window)
    lse = lse.astype(np.float32)
    want, reach = kv8.weigh_ref(c.cache, c.table, c.lens, c.offsets, c.q, lse.astype(np.float64),
                                c.scale, window)
    first = None
    for _ in range(2):
        c.to_gpu()
        lib.kv8_weigh(c.dev, c.batch, c.gpu_q(), torch.from_numpy(lse).cuda(), c.scale, window,
                      c.status)
        assert status(c) == 0
        got = c.dev_arrays()["weight"]
        # exponent's error (scores, the lse's subtraction, the exponential), then fp32 sums
        added = want - c.cache["weight"]
        tol = score_error(D, reach) + 2.0 ** -20 * added + 2.0 ** -22 * want + \
            c.max_new * G * 2.0 ** -24 * added
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
        if first is not None:
            assert np.array_equal(first, got)
        first = got


def test_weights_of_a_row_sum_to_one_per_head(cuda_lib):
    c = Case(41, [777], None, 2, 128, 32, 4)
    c.cache["weight"][:] = 0
    c.to_gpu()
    _, lse = c.attn()
    lib.kv8_weigh(c.dev, c.batch, c.gpu_q(), torch.from_numpy(lse).float().cuda(), c.scale, 0,
                  c.status)
    w = c.dev_arrays()["weight"]
    assert np.allclose(w.sum((0, 2)), 4, atol=1e-4)


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("lens,H,D,P,budget,sink,recent", [
    ([1], 1, 64, 16, 1, 0, 0),
    ([300, 40, 0], 2, 128, 32, 64, 4, 16),
    ([1000], 1, 256, 16, 100, 0, 0),
    ([500, 2500], 2, 64, 128, 300, 2, 100),
    ([4000], 1, 128, 64, 2049, 4, 64),
])
def test_evict(cuda_lib, lens, H, D, P, budget, sink, recent):
    pages = -(-budget // P)
    c = Case(sum(lens) + D, lens, None, H, D, P, spare=pages * len(lens) + 2)
    w = c.cache["weight"]
    w[c.rng.random(w.shape) < 0.3] = 0                     # many equal weights
    w[c.rng.random(w.shape) < 0.2] = 0.5
    c.fix_ranges()
    dst = c.free[:pages * len(lens)].reshape(len(lens), pages).copy()
    c.to_gpu()
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, budget))
    want, kept, new_lens = kv8.evict_ref(c.cache, c.table, c.lens, dst, budget, sink, recent)
    for _ in range(2):
        got_kept, got_lens = lib.kv8_evict(c.dev, c.batch, budget, torch.from_numpy(dst).cuda(),
                                           sink, recent, ws, c.status)
        assert status(c) == 0
        assert np.array_equal(got_kept.cpu().numpy(), kept)
        assert np.array_equal(got_lens.cpu().numpy(), new_lens)
        same(c.dev_arrays(), want)


def test_evict_bad_pages_leave_the_rest(cuda_lib):
    c = Case(51, [100, 90], None, 1, 64, 16, spare=8)
    c.fix_ranges()
    dst = c.free[:8].reshape(2, 4).copy()
    want, kept, _ = kv8.evict_ref(c.cache, c.table, c.lens, dst, 60, 0, 0)
    for n in want:
        for pg in dst[1]:
            want[n][pg] = c.cache[n][pg]
    c.table[1, 3] = -7
    c.to_gpu()
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, 60))
    got, _ = lib.kv8_evict(c.dev, c.batch, 60, torch.from_numpy(dst).cuda(), 0, 0, ws, c.status)
    assert status(c) == lib.STATUS_CODE["W4_ERR_INDEX"]
    assert np.array_equal(got[0].cpu().numpy(), kept[0])
    same(c.dev_arrays(), want)


def test_evicted_cache_is_a_cache(cuda_lib):
    """Attention over the kept tokens equals attention over the same tokens of the source."""
    c = Case(52, [400], None, 2, 128, 16, 4, spare=14)
    c.fix_ranges()
    c.to_gpu()
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, 200))
    dst = torch.from_numpy(c.free[:13][None].copy()).cuda()
    kept, new_lens = lib.kv8_evict(c.dev, c.batch, 200, dst, 4, 8, ws, c.status)
    a = c.dev_arrays()
    q = c.gpu_q()
    batch = lib.KV8Batch(dst, new_lens, max_len=200)
    wa = c.scratch(lib.kv8_attn_workspace_bytes(c.dev, batch, 8))
    out = lib.kv8_attn(c.dev, batch, q, c.scale, workspace=wa, status=c.status)
    assert status(c) == 0
    table = dst.cpu().numpy()
    ref = kv8.attn_ref(a, table, [200], None, c.q, c.scale)
    lse = ref[1]
    check_attn(out.double().cpu().numpy(), lse, ref, 128)
