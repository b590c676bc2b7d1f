"""Forks, growth and compaction of the 8-bit cache's pages against plain simulations: tables,
lengths, references and every byte of the caches have to be equal."""

import numpy as np
import pytest
import torch

from bit_weight_only_gemv_gb300 import lib
from _pages import Pages

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,parents", [
    ([37], [0]),                                   # nothing to do
    ([37], [-1]),                                  # ends
    ([37], [0] * 9),                               # one prompt, nine continuations
    ([32], [0] * 9),                               # its last page is full: nothing to copy
    ([0, 5], [0, 0, 1, 1]),                        # an empty parent
    ([1, 16, 17, 31], [3, 2, 1, 0]),               # everybody moves
    ([1, 16, 17, 31], [1, 1, 3, 3]),
    ([40, 41, 42, 43, 44], [4]),                   # fewer rows: the others end
    ([40, 41, 42, 43, 44], [-1, -1, -1, -1, -1]),
    ([300, 0, 128, 77], [0, 3, 0, 2, 2, 2, -1, 0]),
])
@pytest.mark.parametrize("P,D", [(16, 64), (128, 256)])
def test_fork(cuda_lib, lens, parents, P, D):
    Pages(len(lens), lens, P=P, D=D, layers=2, spare=12).to_gpu(most_rows=16).fork(parents)


def test_fork_of_shared_pages(cuda_lib):
    # rows 0, 1, 2 share whole pages; row 2 was cut back into one of them: it gets its own
    p = Pages(3, [50, 55, 48, 20], share={1: (0, 3), 2: (0, 3), 3: (0, 1)}, layers=3, spare=9)
    p.pool.lens[2] = 40
    p.to_gpu(most_rows=8)
    p.fork([0, 1, 2, 3])
    p.fork([2, 2, 0, 1, 3, 3, -1])


def test_fork_where_something_else_keeps_the_open_page(cuda_lib):
    p = Pages(4, [23, 9], spare=9)
    p.pool.refs[p.pool.table[0, 1]] += 1           # a prefix kept for later
    p.to_gpu(most_rows=4)
    copies = p.fork([0, 1, 0])[3]
    assert [c[0] for c in copies] == [p.pool.table[0, 1]] * 2      # both, and not the kept one


@pytest.mark.parametrize("layered,optional", [(True, True), (False, False)])
def test_fork_strides_and_absent_arrays(cuda_lib, layered, optional):
    Pages(5, [100, 61], P=32, H=3, D=128, layers=4, spare=20, optional=optional).to_gpu(
        layered, most_rows=12).fork([0, 1, 1, 0, 0, 1, 0, 0, 0, 1, 1, 1])


def test_fork_with_just_enough_pages_and_one_too_few(cuda_lib):
    Pages(6, [33, 17], spare=3).to_gpu(most_rows=5).fork([0, 0, 0, 1, 1])
    p = Pages(6, [33, 17], spare=2).to_gpu(most_rows=5)
    assert p.fork([0, 0, 0, 1, 1])[3] is None
    # pages of rows that end in the same call count as free
    p = Pages(6, [33, 17], spare=0).to_gpu(most_rows=5)
    assert p.fork([0, 0, 0])[3] is not None


@pytest.mark.parametrize("spoil", ["parent", "low parent", "length", "negative", "page", "high page"])
def test_fork_of_rows_out_of_bounds(cuda_lib, spoil):
    p = Pages(7, [40, 50, 60, 70], spare=9)
    parents = [0, 0, 2, 2, 1]
    if spoil == "parent":
        parents[1] = 4
    elif spoil == "low parent":
        parents[1] = -2
    elif spoil == "length":
        p.pool.lens[2] = p.pool.table.shape[1] * p.P + 1
    elif spoil == "negative":
        p.pool.lens[2] = -1
    else:
        p.pool.table[2, 1] = -1 if spoil == "page" else p.num
    p.to_gpu(most_rows=8).fork(parents)


def test_many_rows_and_long_rows(cuda_lib):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 60, 4096).tolist()
    p = Pages(8, lens, spare=4096).to_gpu()
    p.fork(rng.integers(-1, 4096, 4096).tolist())
    p.reserve()
    p.compact()
    p = Pages(9, [60000, 3, 50001], D=64, H=1, spare=500, optional=False).to_gpu(most_rows=6)
    p.fork([0, 0, 2, 2, 1, -1])
    p.reserve([0, 400, 900])
    p.compact()


@pytest.mark.parametrize("lens,grow", [
    ([16, 0, 15, 31], None),
    ([16, 0, 15, 31], [1, 0, 1, 33]),
    ([0, 0, 0], [200, 1, 16]),                     # prompts
    ([5], [0]),
    ([40, 40, 40], [-1, 3, 8]),
    ([40, 40, 40], [3, 10 ** 6, 2147483647]),
    ([40, 40, 40], [100, 100, 100]),               # more than there are
])
def test_reserve(cuda_lib, lens, grow):
    p = Pages(10, lens, spare=16, max_pages=20).to_gpu()
    p.reserve(grow)
    p.reserve(None) if int(p.status) == 0 else None


def test_reserve_of_rows_out_of_bounds(cuda_lib):
    p = Pages(11, [40, 16, 32], spare=9)
    p.pool.lens[1] = -1
    p.to_gpu().reserve()


@pytest.mark.parametrize("lens,share,pins,layers", [
    ([5], {}, 0, 1), ([0], {}, 0, 1), ([100, 7, 64], {}, 0, 3), ([100, 70, 64], {1: (0, 4)}, 2, 2),
    ([300, 299, 40, 0, 16], {1: (0, 10), 2: (1, 2)}, 3, 2)])
@pytest.mark.parametrize("spare", [0, 1, 40])
def test_compact(cuda_lib, lens, share, pins, layers, spare):
    p = Pages(12, lens, P=16, D=128, share=share, pins=min(pins, spare), layers=layers,
              spare=spare).to_gpu()
    nt, nr, _ = p.compact()
    # once more: nothing left to move but what something else keeps in the way
    q = Pages(12, lens, P=16, D=128, share=share, pins=0, layers=layers, spare=spare)
    q.pool.table, q.pool.refs = nt.cpu().numpy(), nr.cpu().numpy()
    copies = q.to_gpu().compact()[2]
    assert pins or not copies


@pytest.mark.parametrize("spoil", ["length", "page"])
def test_compact_of_rows_out_of_bounds(cuda_lib, spoil):
    p = Pages(13, [40, 90, 60, 70], share={3: (1, 4)}, spare=30)
    if spoil == "length":
        p.pool.lens[1] = -3
    else:
        p.pool.table[1, 2] = p.num + 5
    p.to_gpu().compact()


@pytest.mark.parametrize("spare", [3000, 9001, 16300, 17000, 70001])
def test_a_pool_of_many_pages(cuda_lib, spare):
    p = Pages(14, [700, 333, 90], H=1, D=64, spare=spare, optional=False).to_gpu(most_rows=8)
    p.fork([0, 0, 1, 1, 2, 2])
    p.reserve()
    p.compact()


def test_calls_in_a_graph(cuda_lib):
    """Fork, then grow, captured once and replayed on other lengths and parents."""
    p = Pages(15, [37, 50, 48, 90], spare=30, layers=2)
    q = Pages(16, [16, 90, 3, 33], spare=30, layers=2, max_pages=p.pool.table.shape[1])
    p.to_gpu()
    parents = torch.tensor([0, 0, 1, 2], dtype=torch.int32, device="cuda")
    nt = torch.full_like(p.table, -9)
    nl, nr = torch.empty_like(p.lens), torch.empty_like(p.refs)
    calls = [lib.bind_kv8_fork(p.dev, p.table, p.lens, p.refs, parents, nt, nl, nr, p.ws, p.status),
             lib.bind_kv8_reserve(nt, nl, nr, p.P, None, p.ws, p.status)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    from oracle import serve
    for case, par in ((p, [0, 0, 1, 2]), (p, [3, -1, 3, 3]), (q, [3, 3, 2, 1])):
        n = min(case.num, p.num)
        assert case.num <= p.num
        refs = np.zeros(p.num, np.int32)
        refs[:n] = case.pool.refs[:n]
        p.table.copy_(torch.from_numpy(case.pool.table))
        p.lens.copy_(torch.from_numpy(case.pool.lens))
        p.refs.copy_(torch.from_numpy(refs))
        parents.copy_(torch.tensor(par, dtype=torch.int32))
        nt.fill_(-9)
        before = [[t.clone() for t in d.tensors] for d in p.dev]
        g.replay()
        torch.cuda.synchronize()
        pool = serve.Pool(case.pool.table, case.pool.lens, refs, p.P)
        table, lens, refs, copies, _ = serve.fork(pool, par, np.full(p.pool.table.shape, -9, np.int32))
        table, lens, refs, _ = serve.reserve(serve.Pool(table, lens, refs, p.P), None)
        assert np.array_equal(nt.cpu().numpy(), table) and np.array_equal(nl.cpu().numpy(), lens)
        assert np.array_equal(nr.cpu().numpy(), refs) and int(p.status) == 0
        for old, d in zip(before, p.dev):
            want = serve.copy_pages(dict(zip(("kc", "vc", "ks", "vs", "ranges", "weight"),
                                             (t.cpu().numpy() for t in old))), copies)
            for name, t in zip(want, d.tensors):
                assert np.array_equal(t.cpu().numpy(), want[name])


def test_as_many_caches_as_a_call_takes(cuda_lib):
    p = Pages(17, [20, 7], H=1, D=64, layers=128, spare=4).to_gpu(most_rows=4)
    p.fork([1, 0, 0, 1])
    p.compact()


def test_copies_follow_the_decision_of_their_call(cuda_lib):
    """What the copying kernel reads is what the deciding one wrote, not what the workspace held before:
    many times, since a load before its time would not show every time."""
    for rep in range(60):
        lens, parents = ([0, 5], [0, 0, 1, 1]) if rep % 2 else ([1, 16, 17, 31], [1, 1, 3, 3])
        p = Pages(rep, lens, layers=2, spare=12).to_gpu(most_rows=4)
        if rep % 3 == 0:
            p.ws[4096:] = 1
        assert p.fork(parents)[3]


@pytest.mark.parametrize("on_a_stream", [False, True])
def test_reserve_brings_its_own_workspace(cuda_lib, on_a_stream):
    p, q = (Pages(18, [16, 0, 15, 31], spare=16, max_pages=20).to_gpu() for _ in range(2))
    p.reserve([1, 40, 0, 2])
    stream = torch.cuda.Stream() if on_a_stream else None
    grow = torch.tensor([1, 40, 0, 2], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    lib.kv8_reserve(q.table, q.lens, q.refs, q.P, grow, stream=stream)
    torch.cuda.synchronize()
    for a, b in ((p.table, q.table), (p.lens, q.lens), (p.refs, q.refs)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        lib.bind_kv8_reserve(q.table, q.lens, q.refs, q.P)


# ---------------------------------------------------------------- refusals where a cluster decides
# (more than 16384 pages, or more than 256 pieces of 128 table entries)
LARGE = {"pages": dict(spare=17000), "pieces": dict(spare=40, max_pages=12000)}


def large(seed, lens, size, H=1, **over):
    return Pages(seed, lens, H=H, D=64, optional=False, **{**LARGE[size], **over})


def spoil(p, how, b, at):
    if how == "length":
        p.pool.lens[b] = p.pool.table.shape[1] * p.P + 1
    elif how == "negative":
        p.pool.lens[b] = -1
    elif how == "page":
        p.pool.table[b, at] = -1
    elif how == "high page":
        p.pool.table[b, at] = p.num


@pytest.mark.parametrize("how,at", [("parent", 0), ("low parent", 0), ("length", 0), ("negative", 0), ("page", 1),
                                    ("high page", 1), ("page", 127), ("high page", 128), ("page", 311),
                                    ("high page", 312)])
@pytest.mark.parametrize("size", ["pages", "pieces", "small"])
def test_fork_of_rows_out_of_bounds_at_any_size(cuda_lib, size, how, at):
    """The last entry of row 2 is number 312, of its third piece."""
    lens = [40, 5000, 5007, 2100]
    p = large(20, lens, size) if size in LARGE else Pages(20, lens, H=1, spare=20, optional=False)
    parents = [0, 0, 2, 2, 1, 3, -1]
    if how == "parent":
        parents[1] = 4
    elif how == "low parent":
        parents[1] = -2
    spoil(p, how, 2, at)
    p.to_gpu(most_rows=8).fork(parents)
    assert int(p.status) == lib.STATUS_CODE["W4_ERR_INDEX"]


@pytest.mark.parametrize("size", ["pages", "pieces"])
def test_fork_with_one_page_too_few_in_a_large_pool(cuda_lib, size):
    """Five rows that end in two pages: three copies.  What is free is kept by something else but for
    three or two pages."""
    for free in (3, 2):
        p = large(21, [33, 17], size)
        unused = np.flatnonzero(p.pool.refs == 0)
        p.pool.refs[unused[:len(unused) - free]] += 1
        copies = p.to_gpu(most_rows=5).fork([0, 0, 0, 1, 1])[3]
        assert (copies is None) == (free == 2)


@pytest.mark.parametrize("size", ["pages", "pieces"])
@pytest.mark.parametrize("grow", [[1, 0, 40, 3000], [-1, 3, 2 ** 31 - 1, 64], None])
@pytest.mark.parametrize("free", [None, 190, 5, 0])
def test_reserve_in_a_large_pool(cuda_lib, size, grow, free):
    p = large(22, [31, 16, 5000, 0], size, max_pages=12000)
    if free is not None:
        unused = np.flatnonzero(p.pool.refs == 0)
        p.pool.refs[unused[:max(0, len(unused) - free)]] += 1
    p.to_gpu().reserve(grow)


@pytest.mark.parametrize("how,at", [("length", 0), ("negative", 0), ("page", 2), ("high page", 200), (None, 0)])
@pytest.mark.parametrize("size", ["pages", "pieces", "small"])
def test_compact_with_pages_that_stay(cuda_lib, size, how, at):
    """Pages that something else keeps, and those of a row out of bounds, among the ones that move."""
    lens, share = [40, 4000, 60, 3000], {3: (1, 100)}
    p = large(23, lens, size, share=share, pins=15) if size in LARGE else \
        Pages(23, lens, H=1, share=share, pins=15, spare=60, optional=False)
    spoil(p, how, 1, at)
    p.to_gpu().compact()
    assert int(p.status) == (lib.STATUS_CODE["W4_ERR_INDEX"] if how else 0)
