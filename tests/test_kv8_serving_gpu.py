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
