"""The 8-bit cache's operators beside one another and beside the products, as a
serving loop runs them."""

import numpy as np
import pytest
import torch

from oracle import kv8
from bit_weight_only_gemv_gb300 import lib
from _kv8 import Case, check_attn

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
