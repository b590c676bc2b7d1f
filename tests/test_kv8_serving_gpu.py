"""The 8-bit cache's operators beside one another and beside the products, as a
serving loop runs them."""

import numpy as np
import pytest
import torch

from oracle import kv8
from bit_weight_only_gemv_gb300 import lib
from _kv8 import Case, check_attn, score_error

pytestmark = pytest.mark.gpu


def status(c):
    torch.cuda.synchronize()
    return int(c.status.item())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_kernels_and_products_as_dependents_of_one_another(cuda_lib, D):
    """Kernels that hold tensor memory, each launched as a dependent of the one before: chunk
    attention, the output product, chunk weights, a product of few rows."""
    n = 64
    c = Case(5 + D, [300], [n], 2, D, 16, 4)
    c.to_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)
    K = 8 * D
    w = lib.quantize(torch.randn((512, K), generator=gen, device="cuda") * K ** -0.5)
    q = c.gpu_q()
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    ws = c.scratch(lib.kv8_attn_workspace_bytes(c.dev, c.batch, 8))
    attn = lib.bind_kv8_attn(c.dev, c.batch, q, c.scale, out, lse=lse, workspace=ws, status=c.status)
    weigh = lib.bind_kv8_weigh(c.dev, c.batch, q, lse, c.scale, status=c.status)
    space = {m: c.scratch(lib.workspace_bytes(m, 512, K)) for m in (n, 8)}
    ys = {m: torch.empty((m, 512), dtype=torch.bfloat16, device="cuda") for m in (n, 8)}

    def product(m):
        lib.gemv(*w, out.view(n, K)[:m], ys[m], workspace=space[m], status=c.status, pdl=True)

    def layer():
        attn(pdl=True)
        product(n)
        weigh(pdl=True)
        product(8)

    layer()
    assert status(c) == 0
    ref = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)
    check_attn(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, D)
    want = [out.clone(), ys[n].clone(), ys[8].clone()]
    grown = c.dev.tensors[5].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            layer()
    graph.replay()
    assert status(c) == 0
    for a, b in zip(want, (out, ys[n], ys[8])):
        assert torch.equal(a, b)
    added = grown.double() - torch.from_numpy(c.cache["weight"]).cuda().double()
    many = c.dev.tensors[5].double() - grown.double()
    # twenty times what one call adds, but for the fp32 sums' roundings
    bound = 21 * 2.0 ** -23 * c.dev.tensors[5].double() + 1e-12
    assert bool((torch.abs(many - 20 * added) <= 20 * bound).all())


def test_one_workspace_for_every_call(cuda_lib):
    """A product, then prompt chunks, single tokens, more sequences, selections and evictions in
    turn on one buffer, zero-filled once: each leaves it ready for the next."""
    def made(seed, lens, news, H, D, P, G, spare=3):
        c = Case(seed, lens, news, H, D, P, G, spare=spare)
        c.fix_ranges()
        c.to_gpu()
        return c, kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale)

    chunk = made(1, [700], [100], 1, 128, 32, 2)
    rows64 = made(2, [900, 260], [90, 33], 2, 64, 16, 3)
    token = made(3, [4000], None, 1, 128, 32, 8, spare=40)
    many = made(4, [int(x) for x in np.random.default_rng(4).integers(1, 1500, 70)], None, 2, 128,
                64, 12)
    wide = made(6, [3000, 2000], None, 2, 256, 16, 4)
    pairs = made(7, [2500, 800], [5, 4], 2, 128, 16, 8)
    sparse = made(5, [6000, 900], None, 2, 64, 16, 4)
    sel_want, n_want = kv8.select_ref(sparse[0].cache, sparse[0].table, sparse[0].lens, sparse[0].q,
                                      200, 1, 1)
    budget = 1100
    dst = token[0].free[:-(-budget // 32)][None].copy()
    cases = (chunk, rows64, token, many, wide, pairs, sparse)
    w = lib.quantize(torch.randn((300, 512), device="cuda") * 0.05)
    x = torch.randn((5, 512), device="cuda").to(torch.bfloat16)
    need = max([lib.kv8_attn_workspace_bytes(c.dev, c.batch, c.H * c.G) for c, _ in cases]
               + [lib.kv8_attn_workspace_bytes(sparse[0].dev, sparse[0].batch, 8, max_sel=200),
                  lib.kv8_select_workspace_bytes(sparse[0].dev, sparse[0].batch),
                  lib.kv8_evict_workspace_bytes(token[0].dev, token[0].batch, budget),
                  lib.workspace_bytes(5, 300, 512)])
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def attend(case, sel=None, n_sel=None, ref=None):
        c = case[0]
        q = c.gpu_q()
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        lib.kv8_attn(c.dev, c.batch, q, c.scale, out, lse, 0, sel, n_sel, ws, c.status)
        assert status(c) == 0
        check_attn(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref or case[1], c.D)

    def choose():
        c = sparse[0]
        sel, n_sel = lib.kv8_select(c.dev, c.batch, c.gpu_q(), 200, 1, 1, ws, c.status)
        assert status(c) == 0
        assert np.array_equal(sel.cpu().numpy(), sel_want)
        assert np.array_equal(n_sel.cpu().numpy(), n_want)
        attend(sparse, sel, n_sel, kv8.attn_ref(c.cache, c.table, c.lens, None, c.q, c.scale, 0,
                                                sel_want, n_want))

    def evict():
        c = token[0]
        want, kept, _ = kv8.evict_ref(c.cache, c.table, c.lens, dst, budget, 4, 16)
        got, _ = lib.kv8_evict(c.dev, c.batch, budget, torch.from_numpy(dst).cuda(), 4, 16, ws,
                               c.status)
        assert status(c) == 0
        assert np.array_equal(got.cpu().numpy(), kept)
        got = c.dev_arrays()
        assert all(np.array_equal(got[n], want[n]) for n in want)

    alone = lib.gemv(*w, x, workspace=torch.zeros_like(ws), status=chunk[0].status)

    def product():
        assert torch.equal(lib.gemv(*w, x, workspace=ws, status=chunk[0].status), alone)

    for step in (product, chunk, token, many, choose, token, evict, wide, product, rows64, sparse,
                 pairs, many, evict, product, token, choose, chunk, wide):
        step() if callable(step) else attend(step)
    assert not bool(ws[:4096].any())


def weigh_chosen(c, q, sel, n_sel, window=0):
    """(weights after one kv8_weigh over the chosen pages, reference, its reach, log-sums)."""
    want_sel, want_n = sel.cpu().numpy(), n_sel.cpu().numpy()
    _, lse, _, _ = kv8.attn_ref(c.cache, c.table, c.lens, c.offsets, c.q, c.scale, window, want_sel,
                                want_n)
    lse = lse.astype(np.float32)
    want, reach = kv8.weigh_ref(c.cache, c.table, c.lens, c.offsets, c.q, lse.astype(np.float64),
                                c.scale, window, want_sel, want_n)
    lib.kv8_weigh(c.dev, c.batch, q, torch.from_numpy(lse).cuda(), c.scale, window, c.status,
                  sel=sel, n_sel=n_sel)
    return want, reach, lse


@pytest.mark.parametrize("lens,H,D,P,G,max_sel,window", [
    ([1], 1, 64, 16, 1, 1, 0),
    ([700, 30, 1, 0], 2, 128, 16, 4, 9, 0),
    ([5000], 2, 256, 16, 8, 40, 0),
    ([1000, 2000], 3, 64, 32, 12, 20, 0),
    ([900, 333], 2, 128, 128, 20, 3, 0),                  # a group of several row tiles
    ([600], 1, 256, 64, 71, 5, 0),
    ([3000, 77], 1, 64, 16, 128, 100, 0),
    ([2000, 500], 2, 128, 32, 3, 16, 300),                # pages before the window add nothing
    ([9000] * 40, 1, 64, 16, 2, 30, 0),                   # more entries than a warp looks at
])
def test_weigh_over_chosen_pages(cuda_lib, lens, H, D, P, G, max_sel, window):
    c = Case(sum(lens) + D, lens, None, H, D, P, G)
    c.fix_ranges()
    c.to_gpu()
    ws = c.scratch(lib.kv8_select_workspace_bytes(c.dev, c.batch))
    q = c.gpu_q()
    sel, n_sel = lib.kv8_select(c.dev, c.batch, q, max_sel, 0, 1, ws, c.status)
    first = None
    for _ in range(2):
        c.to_gpu()
        want, reach, _ = weigh_chosen(c, q, sel, n_sel, window)
        assert status(c) == 0
        got = c.dev_arrays()["weight"]
        # as for the weights over the whole cache: the exponent's error, then fp32 sums
        added = want - c.cache["weight"]
        tol = score_error(D, reach) + 2.0 ** -20 * added + 2.0 ** -22 * want + G * 2.0 ** -24 * added
        assert np.all(np.abs(got - want) <= tol)
        untouched = added == 0
        assert np.array_equal(got[untouched], c.cache["weight"][untouched])
        assert first is None or np.array_equal(first, got)
        first = got


def test_weigh_over_chosen_pages_refusals(cuda_lib):
    """Entries outside the sequence's pages are left out, a count that is none adds nothing, a
    page that is none leaves out its tokens; the rest is right."""
    err = lib.STATUS_CODE["W4_ERR_INDEX"]
    c = Case(33, [100, 90, 80, 70], None, 1, 64, 16, 2)
    c.to_gpu()
    q = c.gpu_q()
    good = torch.tensor([[[0, 3, -1, -1]], [[0, 1, 2, 3]], [[1, 2, 4, -1]], [[2, 3, -1, -1]]],
                        dtype=torch.int32, device="cuda")
    n_good = torch.tensor([[2], [4], [3], [2]], dtype=torch.int32, device="cuda")
    want, reach, lse = weigh_chosen(c, q, good, n_good)
    assert status(c) == 0
    for bad_sel, bad_n, lost in (([0, 3, 7, -1], 3, None), ([0, 3, -2, -1], 3, None),
                                 ([0, 3, -1, -1], 5, 0), ([0, 3, -1, -1], -1, 0)):
        c.to_gpu()
        sel, n_sel = good.clone(), n_good.clone()
        sel[0, 0] = torch.tensor(bad_sel, dtype=torch.int32)
        n_sel[0, 0] = bad_n
        lib.kv8_weigh(c.dev, c.batch, q, torch.from_numpy(lse).cuda(), c.scale, 0, c.status, sel=sel,
                      n_sel=n_sel)
        assert status(c) == err
        got, ref = c.dev_arrays()["weight"], want.copy()
        if lost is not None:
            ref[c.table[lost]] = c.cache["weight"][c.table[lost]]
        assert np.allclose(got, ref, rtol=1e-4, atol=1e-6)
    page = c.table[1, 2]
    c.table[1, 2] = -5
    c.to_gpu()
    lib.kv8_weigh(c.dev, c.batch, q, torch.from_numpy(lse).cuda(), c.scale, 0, c.status, sel=good,
                  n_sel=n_good)
    assert status(c) == err
    ref = want.copy()
    ref[page] = c.cache["weight"][page]
    assert np.allclose(c.dev_arrays()["weight"], ref, rtol=1e-4, atol=1e-6)


def test_decode_loop_weights_and_evictions(cuda_lib):
    """The example's loop step by step: each step adds one per query head to the chosen pages'
    tokens, by the definition, and an eviction keeps what the definition keeps."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "kv8_decode.py")
    spec = importlib.util.spec_from_file_location("kv8_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_tokens=16,
                          max_len=160, budget=96, keep_pages=4, seed=2)
    x = layer.tokens(100 + 70)
    layer.prompt(x[:100])
    before = layer.cache.tensors[5].cpu().numpy()
    assert np.allclose(before.sum((0, 2)), 100 * 4, rtol=1e-4)
    was, lens, table = None, None, None
    for i in range(70):
        evictions = layer.evictions
        layer.step(x[100 + i:101 + i])
        torch.cuda.synchronize()
        assert int(layer.status.item()) == 0
        a = layer.arrays()
        base = before
        if layer.evictions > evictions:
            # the step cut the cache first, then stored its token
            kept_pages = np.array(layer.used[:6], np.int32)[None]
            cut, _, n = kv8.evict_ref(was, table, lens, kept_pages, 96, layer.sink, layer.recent)
            assert n[0] == 96
            for name in ("kc", "vc", "ks", "vs", "ranges"):
                assert np.array_equal(a["cache"][name][kept_pages[0]], cut[name][kept_pages[0]])
            base = cut["weight"]
        page, slot = a["table"][0, (layer.length - 1) // 16], (layer.length - 1) % 16
        base = base.copy()
        base[page, :, slot] = 0                       # the new token starts at nothing
        ref = kv8.attn_ref(a["cache"], a["table"], a["lens"], None, a["q"], layer.scale, 0, a["sel"],
                           a["n_sel"])
        check_attn(a["out"], a["lse"], ref, 64)
        want, reach = kv8.weigh_ref(dict(a["cache"], weight=base), a["table"], a["lens"], None,
                                    a["q"], a["lse"], layer.scale, 0, a["sel"], a["n_sel"])
        got, added = a["cache"]["weight"], want - base
        tol = score_error(64, reach) + 2.0 ** -20 * added + 2.0 ** -22 * want + \
            4 * 2.0 ** -24 * added
        live = a["table"][0, :len(layer.used)]
        assert np.all(np.abs(got - want)[live] <= tol[live])
        assert np.allclose((got.astype(np.float64) - base)[live].sum((0, 2)), 4, rtol=1e-4)
        before, was, lens, table = got, a["cache"], a["lens"], a["table"]
    assert layer.evictions >= 1


@pytest.mark.parametrize("D,P,budget", [(128, 16, 200), (64, 32, 333), (256, 16, 90), (128, 64, 400)])
def test_attention_after_an_eviction_is_that_of_the_kept_tokens(cuda_lib, D, P, budget):
    """Against the source's own tokens at the kept positions.  Blocks have steps s, 2 s and 4 s and
    codes 128 + 4 n, so that rescaling to a block's largest step moves no value."""
    c = Case(52 + D, [700], None, 2, D, P, 4, spare=-(-budget // P) + 1)
    for codes, steps, base in (("kc", "ks", 2.0 ** -9), ("vc", "vs", 2.0 ** -5)):
        c.cache[codes] = (c.rng.integers(-31, 32, c.cache[codes].shape) * 4 + 128).astype(np.uint8)
        c.cache[steps] = (base * 2.0 ** c.rng.integers(0, 3, c.cache[steps].shape)).astype(np.float32)
    c.fix_ranges()
    c.to_gpu()
    pages = -(-budget // P)
    dst = torch.from_numpy(c.free[:pages][None].copy()).cuda()
    ws = c.scratch(max(lib.kv8_evict_workspace_bytes(c.dev, c.batch, budget),
                       lib.kv8_attn_workspace_bytes(c.dev, c.batch, 8)))
    kept, new_lens = lib.kv8_evict(c.dev, c.batch, budget, dst, 4, 8, ws, c.status)
    assert status(c) == 0 and new_lens.tolist() == [budget]
    kept = kept.cpu().numpy()[0]
    batch = lib.KV8Batch(dst, new_lens, max_len=budget)
    lse = torch.full((1, 8), float("nan"), device="cuda")
    out = lib.kv8_attn(c.dev, batch, c.gpu_q(), c.scale, lse=lse, workspace=ws, status=c.status)
    assert status(c) == 0
    # attention of each head over its kept tokens
    ref = [np.zeros((1, 8, D)), np.zeros((1, 8)), np.zeros((1, 8, D)), np.zeros((1, 8))]
    for h in range(2):
        assert kept[h, -1] == 699 and np.all(np.diff(kept[h]) > 0)
        k, v = (kv8.values(c.cache[x], c.cache[y], c.table[0], 700, h)[kept[h]]
                for x, y in (("kc", "ks"), ("vc", "vs")))
        for g in range(4 * h, 4 * h + 4):
            s = c.scale * (k @ c.q[0, g])
            p = np.exp(s - s.max())
            ref[1][0, g] = s.max() + np.log(p.sum())
            p /= p.sum()
            ref[0][0, g], ref[2][0, g] = p @ v, p @ np.abs(v)
            ref[3][0, g] = c.scale * (np.abs(k) @ np.abs(c.q[0, g])).max()
    check_attn(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, D)


@pytest.mark.parametrize("D,G", [(128, 4), (64, 128)])
def test_steps_that_grow_from_call_to_call_in_one_graph(cuda_lib, D, G):
    """Append and attention as dependents of one another, token after token: every call of one
    graph sees the steps and codes that the call before it has just rewritten."""
    B, steps, H = 40, 24, 2
    c = Case(61, [3] * B, None, H, D, 32, G)
    rng = c.rng
    c.fix_ranges()
    table = c.table
    c.to_gpu()
    start = [t.clone() for t in c.dev.tensors]
    calls, outs, rows = [], [], []
    ws = None
    for i in range(steps):
        size = 2.0 ** (i % 7 + i // 3) * 0.01
        k, v = (torch.from_numpy(rng.normal(size=(B, H, D)) * size).cuda().to(torch.bfloat16)
                for _ in range(2))
        q = (torch.from_numpy(rng.normal(size=(B, H * G, D)) / (1 + size)).cuda()).to(torch.bfloat16)
        batch = lib.KV8Batch(c.batch.tensors[0], torch.full((B,), 4 + i, dtype=torch.int32,
                                                            device="cuda"), max_len=4 + steps)
        if ws is None:
            ws = c.scratch(lib.kv8_attn_workspace_bytes(c.dev, batch, H * G))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        calls += [lib.bind_kv8_append(c.dev, batch, k, v, c.status),
                  lib.bind_kv8_attn(c.dev, batch, q, c.scale, out, lse=lse, workspace=ws,
                                    status=c.status)]
        outs.append((out, lse))
        rows.append([x.double().cpu().numpy() for x in (k, v, q)])
    calls[-1]()                                       # (first use of each kernel, outside the graph)
    calls[-2]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call(pdl=True)
    for _ in range(3):
        for t, s in zip(c.dev.tensors, start):
            t.copy_(s)
        graph.replay()
        assert status(c) == 0
        first = [(o.clone(), x.clone()) for o, x in outs]
    cache = c.cache
    for i, (k, v, q) in enumerate(rows):
        lens = np.full(B, 4 + i)
        cache = kv8.append_ref(cache, table, lens, None, k, v)
        some = slice(0, B, 7)                         # (every seventh sequence: the reference is slow)
        ref = kv8.attn_ref(cache, table[some], lens[some], None, q[some], c.scale)
        out, lse = (x.double().cpu().numpy()[some] for x in first[i])
        check_attn(out, lse, ref, D)
    got = c.dev_arrays()
    assert all(np.array_equal(got[n], cache[n]) for n in ("kc", "vc", "ks", "vs", "ranges"))
