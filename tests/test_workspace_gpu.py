"""One zero-filled workspace for products of different shapes in turn."""

import pytest
import torch

from bit_weight_only_gemv_gb300 import lib

pytestmark = pytest.mark.gpu


def made(n, k, m):
    gen = torch.Generator(device="cuda").manual_seed(n + k + m)
    w = lib.quantize(torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5)
    return w, torch.randn((m, k), generator=gen, device="cuda").to(torch.bfloat16)


HEAD = 4096   # W4_WORKSPACE_HEAD of include/w4a16.h


def test_a_product_leaves_the_workspace_ready_for_any_other(cuda_lib):
    """K splits with few and many row tiles, CUDA cores and tensor cores, and balanced runs: the
    bits of a call on a buffer of its own, and a head of zeros behind every call."""
    shapes = [(16, 21504, 1, "cuda"), (300, 512, 5, "tensor"), (8960, 512, 5, "tensor"),
              (43008, 512, 16, "tensor"), (1100, 4096, 1, "cuda"), (96, 8192, 2, "cuda"),
              (200, 2048, 32, "tensor"), (8960, 512, 32, "tensor"), (16, 21504, 1, "cuda")]
    need = [lib.workspace_bytes(m, n, k, path) for n, k, m, path in shapes]
    assert sum(b > 0 for b in need) >= 7
    shared = torch.full((max(need),), 255, dtype=torch.uint8, device="cuda")   # but for the head
    shared[:HEAD] = 0
    for (n, k, m, path), b in zip(shapes, need):
        w, x = made(n, k, m)
        own = torch.zeros(max(16, b), dtype=torch.uint8, device="cuda")
        want = lib.gemv(*w, x, workspace=own, path=path)
        y = torch.full_like(want, float("nan"))
        lib.gemv(*w, x, y, workspace=shared, path=path)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16)), (n, k, m)
        assert not bool(own[:HEAD].any()) and not bool(shared[:HEAD].any()), (n, k, m)
