"""Refusals of the routing, logit and page calls before any launch, their bindings' checks, and the
references against brute force."""

import ctypes
import itertools

import numpy as np
import pytest
import torch

from bit_weight_only_gemv_gb300 import lib
from oracle import serve

P0 = 1 << 20   # an address that is never dereferenced: every call here is refused
ARG, ALIGN, SHAPE, SPACE = 1, 2, 3, 4


def route(ids=P0, weights=P0, logits=P0, kind=0, stride=128, bias=None, rows=1, flags=0, router=True, **over):
    r = dict(experts=128, top_k=8, groups=1, top_groups=1, group_best=2, score=0, renorm=1, scale=1.0)
    r.update(over)
    s = lib.RouterStruct(**r)
    return lib.load().w4_route(ids, weights, ctypes.byref(s) if router else None, logits, kind, stride,
                               bias, rows, None, flags, None)


@pytest.mark.parametrize("over,code", [
    (dict(ids=None), ARG), (dict(weights=None), ARG), (dict(logits=None), ARG), (dict(router=False), ARG),
    (dict(rows=0), ARG), (dict(kind=2), ARG), (dict(flags=2), ARG), (dict(experts=0), ARG),
    (dict(top_k=0), ARG), (dict(groups=0), ARG), (dict(top_groups=0), ARG), (dict(group_best=3), ARG),
    (dict(score=2), ARG), (dict(renorm=2), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(stride=127), ARG), (dict(stride=1 << 32), ARG),
    (dict(experts=1025, stride=2000), SHAPE), (dict(top_k=33), SHAPE), (dict(groups=3), SHAPE),
    (dict(groups=64, top_groups=64), SHAPE), (dict(groups=4, top_groups=5), SHAPE),
    (dict(groups=32, top_groups=1, top_k=5), SHAPE), (dict(experts=4, top_k=5), SHAPE),
    (dict(ids=P0 + 2), ALIGN), (dict(weights=P0 + 1), ALIGN), (dict(bias=P0 + 2), ALIGN),
    (dict(logits=P0 + 1), ALIGN), (dict(logits=P0 + 2, kind=1), ALIGN)])
def test_route_refusals(over, code):
    assert route(**over) == code


def combine(out=P0, y=P0, weights=P0, ids=None, num_experts=0, add=None, rows=1, k=8, N=64, flags=0):
    return lib.load().w4_moe_combine(out, y, weights, ids, num_experts, add, rows, k, N, None, flags, None)


@pytest.mark.parametrize("over,code", [
    (dict(out=None), ARG), (dict(y=None), ARG), (dict(weights=None), ARG), (dict(rows=0), ARG),
    (dict(k=0), ARG), (dict(N=0), ARG), (dict(flags=4), ARG), (dict(ids=P0), ARG), (dict(k=33), SHAPE),
    (dict(out=P0 + 1), ALIGN), (dict(add=P0 + 1), ALIGN), (dict(weights=P0 + 2), ALIGN),
    (dict(ids=P0 + 2, num_experts=4), ALIGN), (dict(rows=2 ** 31 - 1, N=2 ** 20), SHAPE)])
def test_combine_refusals(over, code):
    assert combine(**over) == code


def adjust(logits=P0, kind=0, stride=1000, rows=2, V=1000, flags=0, rules=True, **over):
    r = dict(tokens=P0, lens=P0, prompt=P0, repetition=P0, presence=P0, frequency=P0, bias_ids=P0, bias=P0,
             n_bias=P0, mask=P0, mask_rows=P0, token_stride=64, bias_stride=8, mask_stride=32,
             max_tokens=64, max_bias=8, num_masks=1)
    r.update(over)
    s = lib.LogitRulesStruct(**r)
    return lib.load().w4_logits_adjust(logits, kind, stride, rows, V, ctypes.byref(s) if rules else None,
                                       None, flags, None)


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), ARG), (dict(rules=False), ARG), (dict(rows=0), ARG), (dict(V=0), ARG),
    (dict(kind=3), ARG), (dict(flags=8), ARG), (dict(stride=999), ARG), (dict(tokens=None), ARG),
    (dict(lens=None), ARG), (dict(tokens=None, lens=None), ARG),      # a prompt of no history
    (dict(bias=None), ARG), (dict(bias_ids=None), ARG), (dict(mask=None), ARG), (dict(num_masks=0), ARG),
    (dict(mask_rows=None), ARG),                                      # two rows, one mask
    (dict(max_tokens=-1), ARG), (dict(max_bias=-1), ARG), (dict(token_stride=63), ARG),
    (dict(bias_stride=7), ARG), (dict(mask_stride=31), ARG), (dict(rows=4097), SHAPE),
    (dict(V=(1 << 30) + 1, stride=1 << 31, mask_stride=1 << 30), SHAPE),
    (dict(max_tokens=1 << 19, token_stride=1 << 20), SHAPE), (dict(max_bias=4096, bias_stride=4096), SHAPE),
    (dict(logits=P0 + 1), ALIGN), (dict(logits=P0 + 2, kind=1), ALIGN), (dict(tokens=P0 + 2), ALIGN),
    (dict(mask=P0 + 1), ALIGN), (dict(frequency=P0 + 2), ALIGN)])
def test_adjust_refusals(over, code):
    assert adjust(**over) == code


def pages(name, flags=0, n=2, table=P0, lens=2 * P0, refs=3 * P0, parents=4 * P0, grow=None,
          new_table=5 * P0, new_lens=6 * P0, new_refs=7 * P0, used=8 * P0, batch=3, new_batch=3,
          max_pages=4, num=8, P=16, ws=16 * P0, ws_bytes=1 << 20, second=(), **over):
    c = dict(kc=P0, vc=P0, ks=P0, vs=P0, ranges=P0, weight=P0, num_pages=num, kv_heads=2, page_tokens=P,
             head_dim=64, page_stride=2 * P * 64, head_stride=P * 64)
    c.update(over)
    arr = (lib.KV8CacheStruct * max(1, n))(*[lib.KV8CacheStruct(**{**c, **(dict(second) if i else {})})
                                             for i in range(max(1, min(n, 200)))])
    L = lib.load()
    if name == "fork":
        return L.w4_kv8_fork(new_table, new_lens, new_refs, new_batch, parents, table, lens, refs, batch,
                             max_pages, arr, n, ws, ws_bytes, None, flags, None)
    if name == "reserve":
        return L.w4_kv8_reserve(table, lens, refs, grow, batch, max_pages, num, P, ws, ws_bytes, None,
                                flags, None)
    return L.w4_kv8_compact(new_table, new_refs, used, table, lens, refs, batch, max_pages, arr, n, ws,
                            ws_bytes, None, flags, None)


ALL = ("fork", "reserve", "compact")


@pytest.mark.parametrize("names,over,code", [
    (ALL, dict(table=None), ARG), (ALL, dict(lens=None), ARG), (ALL, dict(refs=None), ARG),
    (ALL, dict(batch=0), ARG), (ALL, dict(max_pages=0), ARG), (ALL, dict(num=0), ARG),
    (ALL, dict(flags=2), ARG), (ALL, dict(batch=4097), SHAPE), (ALL, dict(max_pages=(1 << 26) + 1), SHAPE), (ALL, dict(num=(1 << 30) + 1), SHAPE), (ALL, dict(P=24), SHAPE),
    (ALL, dict(table=P0 + 2), ALIGN), (ALL, dict(ws=P0 + 8), ALIGN), (ALL, dict(ws=None), SPACE),
    (ALL, dict(ws_bytes=4096), SPACE), (("reserve",), dict(grow=P0 + 1), ALIGN),
    (("fork",), dict(parents=None), ARG), (("fork",), dict(new_batch=0), ARG),
    (("fork",), dict(new_batch=4097), SHAPE), (("fork",), dict(new_lens=None), ARG),
    (("fork",), dict(new_lens=2 * P0 + 8), ARG), (("fork",), dict(parents=P0 + 2), ALIGN),
    (("compact",), dict(used=None), ARG), (("compact",), dict(used=P0 + 2), ALIGN),
    (("fork", "compact"), dict(new_table=None), ARG), (("fork", "compact"), dict(new_refs=None), ARG),
    (("fork", "compact"), dict(new_table=P0), ARG), (("fork", "compact"), dict(new_table=P0 + 44), ARG),
    (("fork", "compact"), dict(new_refs=3 * P0), ARG), (("fork", "compact"), dict(n=0), ARG),
    (("fork", "compact"), dict(n=129), SHAPE), (("fork", "compact"), dict(kc=None), ARG),
    (("fork", "compact"), dict(head_dim=96), SHAPE), (("fork", "compact"), dict(kc=P0 + 4), ALIGN),
    (("fork", "compact"), dict(second={"num_pages": 9}), SHAPE),
    (("fork", "compact"), dict(second={"kv_heads": 1}), SHAPE),
    (("fork", "compact"), dict(second={"head_dim": 128, "head_stride": 2048, "page_stride": 4096}), SHAPE)])
def test_page_refusals(names, over, code):
    for name in names:
        assert pages(name, **over) == code, name


def test_page_workspace():
    L = lib.load()
    assert L.w4_kv8_pages_workspace_bytes(0, 8) == 0 and L.w4_kv8_pages_workspace_bytes(8, 0) == 0
    assert L.w4_kv8_pages_workspace_bytes(4097, 8) == 0
    # counts, first rows and three lists of the larger of the two, behind the head
    for b, n in ((1, 1), (4096, 10), (3, 100000)):
        assert L.w4_kv8_pages_workspace_bytes(b, n) >= 4096 + 4 * (b + 2 * n + 3 * max(b, n))


def test_bindings_refuse_what_is_not_on_the_gpu():
    x = torch.zeros((2, 8))
    i = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.route(lib.Router(8, 2), x)
    with pytest.raises(ValueError):
        lib.Router(8, 2, score="relu")
    with pytest.raises(ValueError):
        lib.moe_combine(x.bfloat16(), torch.ones((1, 2)))
    with pytest.raises(ValueError):
        lib.adjust_logits(x, lib.LogitRules())
    with pytest.raises(ValueError):
        lib.LogitRules(tokens=i)
    with pytest.raises(ValueError):
        lib.kv8_reserve(i, i[0], i[0], 16)


# ------------------------------------------------------------------ the references
def test_route_reference_by_brute_force():
    """The chosen set has the largest sum of scores of all sets within all choices of groups."""
    rng = np.random.default_rng(1)
    for _ in range(20):
        x, bias = rng.normal(size=6), rng.normal(size=6) * 0.3
        s = serve.scores(x, True) + bias
        ids, w = serve.route_row(x, bias, 2, 3, 2, 1, True, True, 2.0)
        best = {g: s[2 * g:2 * g + 2].max() for g in range(3)}
        groups = max(itertools.combinations(range(3), 2), key=lambda c: sum(best[g] for g in c))
        can = [e for e in range(6) if e // 2 in groups]
        want = max(itertools.permutations(can, 2), key=lambda c: (s[c[0]], s[c[1]]))
        assert tuple(ids) == want
        assert np.allclose(w, 2.0 * serve.scores(x, True)[ids] / serve.scores(x, True)[ids].sum())
    assert serve.route_row([1, 1, 1], None, 2, 1, 1, 1, False, True, 1.0)[0].tolist() == [0, 1]
    assert serve.route_row([1, np.nan], None, 1, 1, 1, 1, True, True, 1.0) is None


def test_logit_reference_by_hand():
    x = np.array([2.0, -2.0, 1.0, 0.5])
    out, _, named = serve.adjust_row(x, [0, 1, 0, 0], prompt=1, repetition=2.0, presence=0.25, frequency=0.5,
                                     bias=[(2, 9.0), (2, 1.0)], mask=np.array([1, 1, 1, 0], bool))
    assert out.tolist() == [2.0 / 2 - 0.5 * 2 - 0.25, -4.0 - 0.5 - 0.25, 2.0, -np.inf]
    assert named.tolist() == [True, True, True, True]


def test_page_references_keep_their_counts():
    """After any call every page's references are its entries and what keeps it besides."""
    rng = np.random.default_rng(2)
    for trial in range(40):
        P, B, mp, num = 16, 4, 6, 40
        free = list(rng.permutation(num))
        table, lens = np.full((B, mp), -1, np.int32), rng.integers(0, 70, B).astype(np.int32)
        refs = np.zeros(num, np.int32)
        for b in range(B):
            for i in range(-(-int(lens[b]) // P)):
                table[b, i] = free.pop()
                refs[table[b, i]] += 1
        kept = [free.pop() for _ in range(2)]
        refs[kept] += 1

        def counted(table, lens):
            n = np.zeros(num, int)
            n[kept] += 1
            for b in range(len(lens)):
                for p in table[b, :-(-int(lens[b]) // P)]:
                    n[p] += 1
            return n

        pool = serve.Pool(table, lens, refs, P)
        t2, l2, r2, copies, errors = serve.fork(pool, rng.integers(-1, B, 5).tolist(),
                                                np.full((5, mp), -1, np.int32))
        assert not errors and np.array_equal(r2, counted(t2, l2))
        ends = [t2[b, -(-int(n) // P) - 1] for b, n in enumerate(l2) if n % P]
        assert all(r2[p] == 1 for p in ends)
        t3, l3, r3, errors = serve.reserve(serve.Pool(t2, l2, r2, P), None)
        assert not errors and np.array_equal(r3, counted(t3, l3))
        t4, r4, used, moves, _ = serve.compact(serve.Pool(t3, l3, r3, P), t3)
        assert np.array_equal(r4, counted(t4, l3)) and used == np.nonzero(r4)[0].max() + 1
        back = {b: a for a, b, _ in moves}
        for b, n in enumerate(l3):
            k = -(-int(n) // P)
            assert [back.get(p, p) for p in t4[b, :k]] == t3[b, :k].tolist()


@pytest.mark.parametrize("name,over", [
    ("fork", dict(new_lens=4 * P0)),                    # the parents' own array
    ("fork", dict(new_lens=4 * P0 + 8)), ("fork", dict(new_table=4 * P0 - 44)),
    ("fork", dict(new_refs=4 * P0 - 28)), ("fork", dict(new_lens=3 * P0 + 28)),
    ("fork", dict(new_refs=2 * P0 + 8)), ("fork", dict(new_table=2 * P0 - 44)), ("fork", dict(new_lens=P0 + 44)),
    ("fork", dict(new_lens=5 * P0)), ("fork", dict(new_refs=5 * P0 + 44)), ("fork", dict(new_lens=7 * P0 + 28)),
    ("compact", dict(used=P0)), ("compact", dict(used=2 * P0 + 8)), ("compact", dict(used=3 * P0 + 28)),
    ("compact", dict(used=5 * P0 + 44)), ("compact", dict(used=7 * P0)), ("compact", dict(new_table=2 * P0)),
    ("compact", dict(new_refs=2 * P0 + 8)), ("compact", dict(new_refs=5 * P0 + 44))])
def test_page_outputs_overlap_nothing(name, over):
    """An output that lies on an input or on another output, by one word at the least: a large pool's
    CTAs would read the one while others write the other.  (Without a workspace nothing ever starts.)"""
    assert pages(name, ws_bytes=0, **over) == ARG


@pytest.mark.parametrize("name,over", [
    ("fork", dict(new_lens=4 * P0 + 12)), ("fork", dict(new_lens=4 * P0 - 12)), ("fork", dict(new_table=4 * P0 - 48)),
    ("fork", dict(new_refs=2 * P0 + 12)), ("fork", dict(new_refs=5 * P0 + 48)), ("fork", dict(new_lens=7 * P0 + 32)),
    ("compact", dict(used=P0 - 4)), ("compact", dict(used=2 * P0 + 12)), ("compact", dict(used=5 * P0 + 48)),
    ("compact", dict(new_refs=3 * P0 + 32))])
def test_page_outputs_may_touch_others(name, over):
    """Arrays end to end, as in one allocation (the call is refused for its workspace, which comes last)."""
    assert pages(name, ws_bytes=0, **over) == SPACE
