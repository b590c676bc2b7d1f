"""More of the 8-bit cache's operators on the GPU: many sequences, wide groups
over chosen pages, addresses past 32 bits, one workspace for changing lengths,
captured graphs, and a decode loop that uses them together."""

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


def weigh_and_check(c, window=0):
    _, lse, _, _ = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale, window)
    lse = lse.astype(np.float32)
    want, reach = kv8.weigh_ref(c.cache, c.table, c.lens, c.offsets, c.q, lse.astype(np.float64),
                                c.scale, window)
    lib.kv8_weigh(c.dev, c.batch, c.gpu_q(), torch.from_numpy(lse).cuda(), c.scale, window, c.status)
    assert status(c) == 0
    got = c.dev_arrays()["weight"]
    added = want - c.cache["weight"]
    tol = score_error(c.D, reach) + 2.0 ** -20 * added + 2.0 ** -22 * want + \
        c.max_new * c.G * 2.0 ** -24 * added
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("B,news,G,window", [(33, False, 2, 0), (300, False, 8, 40),
                                             (40, True, 3, 0), (290, True, 6, 25)])
def test_many_sequences(cuda_lib, B, news, G, window):
    """More sequences than a warp or a CTA looks at in one go, empty ones among them."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B)
    lens[rng.random(B) < 0.1] = 0
    n = [int(min(x, rng.integers(0, 9))) for x in lens] if news else None
    c = Case(B + 1, [int(x) for x in lens], n, 2, 64, 16, G)
    c.to_gpu()
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale, window)
    out, lse = c.attn(window)
    assert status(c) == 0
    check_attn(out, lse, ref, 64)
    weigh_and_check(c, window)


def test_wide_group_over_chosen_pages(cuda_lib):
    """More query heads than one row tile holds, with a selection of each kind of length."""
    for D in (64, 128, 256):
        c = Case(60 + D, [700, 30, 1], None, 2, D, 16, 20)
        c.fix_ranges()
        c.to_gpu()
        ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
        sel, n_sel = lib.kv8_select(c.dev, c.batch, c.gpu_q(), 9, 1, 1, ws, c.status)
        want, n_want = kv8.select_ref(c.cache, c.table, c.lens, c.q, 9, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(n_sel.cpu().numpy(), n_want)
        out, lse = c.attn(sel=sel, n_sel=n_sel)
        assert status(c) == 0
        check_attn(out, lse, kv8.attn_ref(c.cache, c.table, c.lens, None, c.q, c.scale, 0, want,
                                          n_want), D)


@pytest.mark.parametrize("news", [None, [40]])
def test_pages_gigabytes_apart(cuda_lib, news):
    """Three pages 2.5 GB from one another: offsets past 32 bits in every kernel."""
    c = Case(71, [40], news, 2, 128, 16, 4, spare=2)
    c.fix_ranges()
    c.to_gpu()
    pages = c.cache["kc"].shape[0]
    stride = 5 << 29
    store = [torch.empty(stride * (pages - 1) + 2 * 16 * 128, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    far = [torch.as_strided(s, (pages, 2, 16, 128), (stride, 16 * 128, 128, 1)) for s in store]
    far[0].copy_(c.dev.tensors[0])
    far[1].copy_(c.dev.tensors[1])
    c.dev = lib.KV8Cache(far[0], far[1], *c.dev.tensors[2:4], ranges=c.dev.tensors[4],
                         weight=c.dev.tensors[5])
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    out, lse = c.attn()
    assert status(c) == 0
    check_attn(out, lse, ref, 128)
    weigh_and_check(c)
    # the ranges as the writer keeps them: over the tokens before the new ones
    c.fix_ranges([40 - c.rows])
    c.dev.tensors[4].copy_(torch.from_numpy(c.cache["ranges"]))
    k, v = (bf16_round(c.rng.normal(size=(c.rows, 2, 128))) for _ in range(2))
    want = kv8.append_ref(c.dev_arrays(), c.table, c.lens, c.offsets, k, v)
    lib.kv8_append(c.dev, c.batch, *(torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (k, v)),
                   c.status)
    assert status(c) == 0
    got = c.dev_arrays()
    assert all(np.array_equal(got[n], want[n]) for n in want)
    if news is None:
        dst = c.free[:1][None].copy()
        want, kept, _ = kv8.evict_ref(got, c.table, c.lens, dst, 14, 2, 4)
        ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, 14))
        lib.kv8_evict(c.dev, c.batch, 14, torch.from_numpy(dst).cuda(), 2, 4, ws, c.status)
        assert status(c) == 0
        got = c.dev_arrays()
        assert all(np.array_equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("news", [None, [9, 20, 4]])
def test_one_workspace_for_changing_lengths(cuda_lib, news):
    """A bound call replayed from a graph while the lengths on the device change."""
    full = [400, 333, 250]
    c = Case(81, full, news, 2, 128, 32, 3)
    c.to_gpu()
    q = c.gpu_q()
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    ws = c.scratch(lib.kv8_attn_workspace_bytes(c.dev, c.batch, 6))
    call = lib.bind_kv8_attn(c.dev, c.batch, q, c.scale, out, lse=lse, workspace=ws, status=c.status)
    call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for lens in (full, [20, 20, 20], [100, 333, 21], [9, 400 // 2, 250], full):
        c.lens = np.array(lens, np.int32)
        c.batch.tensors[1].copy_(torch.from_numpy(c.lens))
        graph.replay()
        assert status(c) == 0
        ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
        check_attn(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, 128)


@pytest.mark.parametrize("n,max_sel", [(20000, 77), (300000, 1000)])
def test_select_from_long_lists(cuda_lib, n, max_sel):
    """Pages past what the choosing CTA holds in registers (16 tokens each)."""
    c = Case(91, [n], None, 1, 64, 16, 2)
    c.fix_ranges()
    c.to_gpu()
    ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
    sel, n_sel = lib.kv8_select(c.dev, c.batch, c.gpu_q(), max_sel, 2, 3, ws, c.status)
    want, n_want = kv8.select_ref(c.cache, c.table, c.lens, c.q, max_sel, 2, 3)
    assert status(c) == 0
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(n_sel.cpu().numpy(), n_want)


@pytest.mark.parametrize("n,budget", [(9000, 1000), (17000, 3000)])
def test_evict_from_long_lists(cuda_lib, n, budget):
    pages = -(-budget // 16)
    c = Case(92, [n], None, 1, 64, 16, spare=pages)
    c.cache["weight"][c.rng.random(c.cache["weight"].shape) < 0.5] = 0.25
    c.fix_ranges()
    dst = c.free[:pages][None].copy()
    c.to_gpu()
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, budget))
    want, kept, _ = kv8.evict_ref(c.cache, c.table, c.lens, dst, budget, 4, 32)
    got_kept, _ = lib.kv8_evict(c.dev, c.batch, budget, torch.from_numpy(dst).cuda(), 4, 32, ws,
                                c.status)
    assert status(c) == 0
    assert np.array_equal(got_kept.cpu().numpy(), kept)
    got = c.dev_arrays()
    assert all(np.array_equal(got[x], want[x]) for x in want)


def test_evict_orders_special_weights(cuda_lib):
    """A NaN counts as the largest, infinity next, -0 equals 0 (the lower position first)."""
    c = Case(93, [32], None, 1, 64, 16, spare=1)
    w = np.full(32, -1.0, np.float32)
    w[5], w[9], w[11], w[20], w[3] = -0.0, 0.0, np.nan, np.inf, 0.5
    for i in range(2):
        c.cache["weight"][c.table[0, i], 0] = w[16 * i:16 * i + 16]
    c.to_gpu()
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, 4))
    kept, _ = lib.kv8_evict(c.dev, c.batch, 4, torch.from_numpy(c.free[:1][None].copy()).cuda(),
                            0, 0, ws, c.status)
    assert status(c) == 0
    assert kept.flatten().tolist() == [3, 5, 11, 20]


def test_refused_outputs_stay_unwritten(cuda_lib):
    """A sequence over its bound: selection and eviction leave its outputs alone."""
    err = lib.STATUS_CODE["W4_ERR_INDEX"]
    c = Case(94, [64, 64], None, 1, 64, 16, 2, spare=8)
    c.fix_ranges()
    c.to_gpu()
    c.batch.tensors[1][1] = 65
    sel = torch.full((2, 1, 3), -9, dtype=torch.int32, device="cuda")
    n_sel = torch.full((2, 1), -9, dtype=torch.int32, device="cuda")
    ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
    lib.bind_kv8_select(c.dev, c.batch, c.gpu_q(), sel, n_sel, 1, 1, ws, c.status)()
    assert status(c) == err
    assert sel[1].flatten().tolist() == [-9] * 3 and n_sel.flatten().tolist() == [3, -9]
    c.status.zero_()
    kept = torch.full((2, 1, 20), -9, dtype=torch.int32, device="cuda")
    new_lens = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    dst = torch.from_numpy(c.free[:4].reshape(2, 2).copy()).cuda()
    before = c.dev_arrays()
    ws = c.scratch(lib.kv8_evict_workspace_bytes(c.dev, c.batch, 20))
    lib.bind_kv8_evict(c.dev, c.batch, dst, kept, new_lens, 0, 0, ws, c.status)()
    assert status(c) == err
    assert kept[1].flatten().tolist() == [-9] * 20 and new_lens.tolist() == [20, -9]
    after = c.dev_arrays()
    for pg in dst[1].tolist():
        assert all(np.array_equal(before[n][pg], after[n][pg]) for n in before)


def test_decode_loop_example(cuda_lib):
    """The example's loop: products, cache and attention together, against the same steps in
    fp64 on the cache's own contents."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "kv8_decode.py")
    spec = importlib.util.spec_from_file_location("kv8_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_tokens=16,
                          max_len=200, budget=96, keep_pages=4, seed=1)
    prompt, steps = 100, 120                      # past max_len: one eviction at least
    x = layer.tokens(prompt + steps)
    layer.prompt(x[:prompt])
    for i in range(steps):
        layer.step(x[prompt + i:prompt + i + 1])
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    assert layer.evictions >= 1
    a = layer.arrays()
    ref = kv8.attn_ref(a["cache"], a["table"], a["lens"], None, a["q"], layer.scale, 0, a["sel"],
                       a["n_sel"])
    check_attn(a["out"], ref[1], ref, 64)


@pytest.mark.parametrize("news,D", [(None, 128), ([5, 9], 64), ([30, 20], 128), ([70, 90], 256)])
def test_window_beyond_every_length(cuda_lib, news, D):
    """A window as long as the type allows is none at all."""
    c = Case(71, [300, 190], news, 2, D, 16, 4)
    c.to_gpu()
    plain = c.attn()
    wide = c.attn(window=2 ** 31 - 1)
    assert status(c) == 0
    assert np.array_equal(plain[0], wide[0]) and np.array_equal(plain[1], wide[1])
    got = []
    for window in (0, 2 ** 31 - 1):
        c.to_gpu()
        lib.kv8_weigh(c.dev, c.batch, c.gpu_q(), torch.from_numpy(plain[1]).float().cuda(), c.scale,
                      window, c.status)
        assert status(c) == 0
        got.append(c.dev_arrays()["weight"])
    assert np.array_equal(got[0], got[1])


@pytest.mark.parametrize("G", [3, 5, 48, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weigh_many_rows_of_odd_groups(cuda_lib, G, D):
    """Query tiles of whole tokens: groups that do not divide 128, several units a CTA."""
    c = Case(72 + G, [40, 700, 0, 333, 129], [40, 3, 0, 33, 1], 2, D, 32, G)
    c.to_gpu()
    weigh_and_check(c)
    c.to_gpu()
    weigh_and_check(c, 100)


@pytest.mark.parametrize("news", [None, [9, 4], [60, 33]])
@pytest.mark.parametrize("D", [64, 256])
def test_query_rows_with_gaps(cuda_lib, news, D):
    """A row stride that no head's size divides: the same bits as dense rows."""
    c = Case(75, [200, 90], news, 2, D, 16, 3)
    c.to_gpu()
    q = c.gpu_q()
    n = q.shape[1] * D
    wide = torch.full((q.shape[0], n + 8), float("nan"), dtype=q.dtype, device=q.device)
    wide[:, :n] = q.view(-1, n)
    gaps = wide[:, :n].unflatten(1, (q.shape[1], D))
    dense, spread = c.attn(), c.attn(q=gaps)
    assert status(c) == 0
    assert np.array_equal(dense[0], spread[0]) and np.array_equal(dense[1], spread[1])
    got = []
    for x in (q, gaps):
        c.to_gpu()
        lib.kv8_weigh(c.dev, c.batch, x, torch.from_numpy(dense[1]).float().cuda(), c.scale, 0,
                      c.status)
        assert status(c) == 0
        got.append(c.dev_arrays()["weight"])
    assert np.array_equal(got[0], got[1])
