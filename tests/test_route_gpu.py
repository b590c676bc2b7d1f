"""Routing and expert sums on the GPU against fp64 references."""

import numpy as np
import pytest
import torch

from bit_weight_only_gemv_gb300 import lib
from oracle import serve

pytestmark = pytest.mark.gpu

POISON = -77


def run(x, k, groups=1, top_groups=1, best=2, score="softmax", renorm=True, scale=1.0, bias=None,
        dtype=torch.float32, pad=0):
    """(ids, weights, status) with outputs poisoned before; x fp64 [T, E]; the logits' fp64 values
    as the type holds them."""
    T, E = x.shape
    full = torch.full((T, E + pad), float("nan"), dtype=dtype, device="cuda")
    logits = full[:, :E]
    logits.copy_(torch.from_numpy(x.astype(np.float32)))
    router = lib.Router(E, k, groups, top_groups, best, score, renorm, scale)
    ids = torch.full((T, k), POISON, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), float(POISON), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    lib.bind_route(router, logits, ids, weights, b, status)()
    torch.cuda.synchronize()
    held = logits.double().cpu().numpy()
    return ids.cpu().numpy(), weights.double().cpu().numpy(), int(status), held


def check(x, k, groups=1, top_groups=1, best=2, score="softmax", renorm=True, scale=1.0, bias=None,
          dtype=torch.float32, pad=0):
    """Ids equal; weights within: each score 2^-21 (2^-17 with a softmax's sum), the sum of k of
    them (k - 1) 2^-24 and as much as its terms, quotient and scale 2^-21; an exponential's
    argument is off by 2^-24 of the logits' spread."""
    ids, w, status, held = run(x, k, groups, top_groups, best, score, renorm, scale, bias, dtype, pad)
    b = None if bias is None else bias.astype(np.float32).astype(np.float64)
    refused = False
    for t in range(len(x)):
        ref = serve.route_row(held[t], b, k, groups, top_groups, best, score == "sigmoid", renorm, scale)
        if ref is None:
            refused = True
            assert (ids[t] == POISON).all() and (w[t] == POISON).all()
            continue
        assert np.array_equal(ids[t], ref[0]), (t, ids[t], ref[0])
        chosen = held[t][ref[0]]
        top = held[t].max()
        fin = chosen[np.isfinite(chosen)]
        spread = max([0.0, *(abs(np.clip(v, -110, 110)) for v in fin),
                      *(min(top - v, 110.0) for v in fin if np.isfinite(top))])
        tol = 2.0 ** -16 + k * 2.0 ** -23 + 2.0 ** -23 * spread
        assert np.all(np.abs(w[t] - ref[1]) <= tol * np.abs(ref[1]) + scale * 2.0 ** -125), \
            (t, w[t], ref[1])
    assert status == (lib.STATUS_CODE["W4_ERR_VALUE"] if refused else 0)


SHAPES = [  # T, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 5, 3, 5, 4), (1, 128, 8, 1, 1), (70, 128, 8, 1, 1),
    (33, 60, 6, 4, 2), (17, 64, 32, 2, 2), (9, 96, 4, 8, 3), (40, 256, 8, 8, 4), (21, 160, 6, 8, 1),
    (12, 257, 10, 1, 1), (6, 512, 16, 32, 5), (5, 1000, 7, 10, 9), (4, 1024, 32, 32, 31),
    (1000, 24, 2, 3, 1)]


@pytest.mark.parametrize("T,E,k,G,tg", SHAPES)
@pytest.mark.parametrize("score,bias,best,dtype", [
    ("softmax", False, 1, torch.bfloat16), ("softmax", True, 2, torch.float32),
    ("sigmoid", False, 2, torch.bfloat16), ("sigmoid", True, 1, torch.float32),
    ("sigmoid", True, 2, torch.bfloat16), ("softmax", False, 2, torch.float32)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(cuda_lib, T, E, k, G, tg, score, bias, best, dtype, renorm):
    rng = np.random.default_rng(T * 1000 + E)
    x = rng.normal(size=(T, E)) * 2
    b = rng.normal(size=E) * 0.1 if bias else None
    check(x, k, G, tg, best, score, renorm, 2.5, b, dtype, pad=3 if E % 2 else 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,tg", [(256, 8, 1, 1), (256, 8, 8, 4), (60, 6, 4, 2), (1024, 16, 1, 1)])
def test_scores_nearer_than_32_bits_can_tell(cuda_lib, score, E, k, G, tg):
    """Biases that bring every score to nearly the same sum: the choice is that of 64 bits."""
    rng = np.random.default_rng(E + G)
    x = np.tile(rng.normal(size=(1, E)), (6, 1)).astype(np.float32).astype(np.float64)
    s = serve.scores(x[0], score == "sigmoid")
    bias = (0.75 - s).astype(np.float32)
    check(x, k, G, tg, 2, score, True, 1.0, bias)
    bias[::3] += np.float32(2.0 ** -20)
    check(x, k, G, tg, 1, score, False, 1.0, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
def test_ties_go_to_the_lowest_number(cuda_lib, score, bias):
    rng = np.random.default_rng(3)
    b = None if bias is None else np.full(128, bias)
    x = rng.integers(-2, 3, (50, 128)).astype(np.float64)      # five values
    x[0] = 0.0
    x[1] = np.where(np.arange(128) % 2, 0.0, -0.0)             # zeros of both signs are equal
    check(x, 8, 1, 1, 2, score, True, 1.0, b, torch.bfloat16)
    check(x, 8, 8, 3, 2, score, True, 1.0, b, torch.bfloat16)
    check(x, 8, 8, 3, 1, score, False, 1.0, b)


def test_extreme_logits(cuda_lib):
    rng = np.random.default_rng(4)
    x = rng.normal(size=(8, 64))
    x[0, :40] = -np.inf
    x[1] = -np.inf
    x[1, 5] = 1.0                             # one expert left: the others have scores of 0
    x[2] *= 60                                # sigmoids that are 1 in 32 bits, in the logits' order
    x[3] = x[3] - 300                         # scores below the smallest number, weights that are not
    x[4] = 3e38
    x[5, 7] = -3e38
    x[6] = -200 + np.arange(64) / 8
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check(x, 6, 1, 1, 2, score, renorm, 1.0)
    check(np.full((2, 16), -np.inf), 4, score="sigmoid")       # weights of 0
    check(np.where(np.arange(64) % 3 == 0, -np.inf, x), 30, 4, 3, 1, "softmax", True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_refused_tokens_stay_unwritten(cuda_lib, score):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(9, 96))
    x[1, 3] = np.nan
    x[4] = np.nan
    x[6, 95] = np.inf
    x[8] = -np.inf
    check(x, 5, score=score)
    b = np.zeros(96)
    b[17] = np.inf
    check(rng.normal(size=(3, 96)), 5, score=score, bias=b)


def test_many_tokens(cuda_lib):
    """A prompt of 5003 tokens: each row as it is alone."""
    rng = np.random.default_rng(6)
    x = rng.normal(size=(5003, 256))
    b = rng.normal(size=256) * 0.05
    ids, w, status, _ = run(x, 8, 8, 4, 2, "sigmoid", True, 2.5, b, torch.bfloat16)
    assert status == 0
    for t in (0, 1, 2500, 5001, 5002):
        i1, w1, _, _ = run(x[t:t + 1], 8, 8, 4, 2, "sigmoid", True, 2.5, b, torch.bfloat16)
        assert np.array_equal(i1[0], ids[t]) and np.array_equal(w1[0], w[t])
    part = rng.integers(0, 5003, 60)
    check(x[part], 8, 8, 4, 2, "sigmoid", True, 2.5, b, torch.bfloat16)


@pytest.mark.parametrize("T,k,N,add,shift", [
    (1, 8, 2816, False, 0), (1, 1, 1, True, 0), (5, 3, 64, True, 0), (7, 11, 351, True, 0),
    (3, 32, 1000, False, 0), (300, 8, 704, True, 0), (2, 8, 4096, False, 1), (9, 2, 8, True, 3)])
def test_combine(cuda_lib, T, k, N, add, shift):
    """fp32 sums of k + 1 terms, (k + 1) 2^-24 of their magnitudes, then half a bf16 step, 2^-8."""
    rng = np.random.default_rng(T + k + N)

    def dev(shape):      # `shift` elements past a 16-byte boundary
        t = torch.zeros(int(np.prod(shape)) + shift, dtype=torch.bfloat16, device="cuda")[shift:]
        return t.view(shape).copy_(torch.from_numpy(rng.normal(size=shape).astype(np.float32)))

    y, out = dev((T * k, N)), dev((T, N))
    a = dev((T, N)) if add else None
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    ids = torch.from_numpy(rng.integers(0, 9, (T, k)).astype(np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref, size = serve.combine(y.double().cpu().numpy(), w.double().cpu().numpy(),
                              None if a is None else a.double().cpu().numpy())
    tol = (k + 1) * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(ref)
    for i in (None, ids):
        out.fill_(float("nan"))
        lib.moe_combine(y, w, out, a, i, 9, status)
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)
    if add:      # in place
        lib.moe_combine(y, w, a, a, ids, 9, status)
        assert torch.equal(a, out)
    assert int(status) == 0


def test_combine_leaves_tokens_of_bad_ids(cuda_lib):
    y = torch.ones((12, 40), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((4, 3), device="cuda")
    ids = torch.tensor([[0, 1, 2], [3, 4, 5], [0, -1, 2], [5, 5, 6]], dtype=torch.int32, device="cuda")
    out = torch.full((4, 40), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.moe_combine(y, w, out, None, ids, 6, status)
    assert int(status) == lib.STATUS_CODE["W4_ERR_INDEX"]
    assert out[:, 0].tolist() == [3.0, 3.0, 9.0, 9.0] and (out == out[:, :1]).all()


def test_combine_keeps_what_is_not_finite(cuda_lib):
    y = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")
    y[0, 1], y[1, 2], y[2, 3] = float("inf"), float("nan"), 3e38
    w = torch.tensor([[0.5, 0.5], [1.0, 0.0]], device="cuda")
    out = lib.moe_combine(y, w).double().cpu().numpy()
    assert out[0, 1] == np.inf and np.isnan(out[0, 2]) and out[0, 3] == 0
    assert np.isfinite(out[1]).all()


@pytest.mark.parametrize("E,k,G,tg", [(256, 8, 8, 4), (256, 8, 1, 1), (256, 3, 8, 1), (256, 8, 4, 1), (256, 8, 8, 1),
                                      (128, 8, 1, 1), (128, 5, 2, 1), (64, 6, 1, 1), (64, 8, 8, 5)])
@pytest.mark.parametrize("score,bias,best,dtype", [
    ("softmax", False, 1, torch.bfloat16), ("softmax", True, 2, torch.float32),
    ("sigmoid", True, 2, torch.bfloat16), ("sigmoid", False, 2, torch.float32),
    ("sigmoid", False, 1, torch.bfloat16)])
def test_many_tokens_as_each_alone(cuda_lib, E, k, G, tg, score, bias, best, dtype):
    """4099 tokens in one call, the ids of calls of 1000, and of the reference for some: near scores,
    ties, extremes and refused tokens among them."""
    rng = np.random.default_rng(E + k + G)
    T = 4099
    x = rng.normal(size=(T, E)) * 2
    x[5] = x[5, 0]                                     # all equal
    x[100:140] = np.round(x[100:140])                  # many ties
    x[200, 3] = np.nan
    x[201, :] = -np.inf
    x[202, 7] = np.inf
    x[300:310, E // 2:] = -np.inf
    x[400:420] *= 30
    x[500:520, :E // 16] += 12                         # one lane's experts all the best
    x[T - 1, 1] = np.nan
    b = rng.normal(size=E) * 0.05 if bias else None
    if bias:                                           # scores that 32 bits cannot tell apart
        xf = torch.from_numpy(x[600].astype(np.float32)).to(dtype).double().numpy()
        s = serve.scores(xf, score == "sigmoid")
        b = np.float32(np.median(s + b)) - s
        b += rng.normal(size=E) * 0.03 * (rng.random(E) < 0.8)
    renorm = k != 6 and G != 1
    ids, w, status, held = run(x, k, G, tg, best, score, renorm, 1.0, b, dtype)
    assert status == lib.STATUS_CODE["W4_ERR_VALUE"]
    for t0 in range(0, T, 1000):
        i1, w1, _, _ = run(x[t0:t0 + 1000], k, G, tg, best, score, renorm, 1.0, b, dtype)
        assert np.array_equal(i1, ids[t0:t0 + 1000])
        assert np.array_equal(w1, w[t0:t0 + 1000])
        # (the same bits, however many tokens a call has)
    part = np.r_[0:10, 100:105, 198:204, 300:303, 400:405, 500:505, 598:603, T - 4:T]
    b64 = None if b is None else b.astype(np.float32).astype(np.float64)
    for t in part:
        ref = serve.route_row(held[t], b64, k, G, tg, best, score == "sigmoid", renorm, 1.0)
        if ref is None:
            assert (ids[t] == POISON).all() and (w[t] == POISON).all()
        else:
            assert np.array_equal(ids[t], ref[0]), (t, ids[t], ref[0])


@pytest.mark.parametrize("E,pad,dtype", [(256, 1, torch.bfloat16), (128, 2, torch.float32), (250, 0, torch.bfloat16)])
def test_many_tokens_at_any_stride(cuda_lib, E, pad, dtype):
    rng = np.random.default_rng(E)
    x, b = rng.normal(size=(4200, E)), rng.normal(size=E) * 0.05
    ids, w, status, held = run(x, 6, 2, 1, 1, "sigmoid", True, 1.0, b, dtype, pad)
    assert status == 0
    for t in (0, 1, 2047, 4198, 4199):
        ref = serve.route_row(held[t], b.astype(np.float32).astype(np.float64), 6, 2, 1, 1, True, True, 1.0)
        assert np.array_equal(ids[t], ref[0]) and np.allclose(w[t], ref[1], rtol=2.0 ** -18, atol=0)
    check(x[4100:], 6, 2, 1, 1, "sigmoid", True, 1.0, b, dtype, pad)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [20, 60, 1000])
@pytest.mark.parametrize("T,E,G,tg,k", [(300, 256, 8, 4, 8), (4099, 256, 8, 4, 8), (4099, 128, 4, 2, 6),
                                        (200, 512, 16, 5, 16), (200, 1024, 8, 2, 3)])
def test_groups_by_their_best_logit_alone(cuda_lib, score, spread, T, E, G, tg, k):
    """Scores of 1 or of 0, in 64 bits too, do not make groups equal whose logits are not: with
    group_best 1 and no bias the groups' order is that of their largest logits, in either type."""
    rng = np.random.default_rng(spread + E)
    x = torch.from_numpy(rng.normal(size=(T, E)) * spread).bfloat16().double().numpy()   # both types hold it
    got = {}
    for dtype in (torch.float32, torch.bfloat16):
        got[dtype], _, status, held = run(x, k, G, tg, 1, score, True, 1.0, None, dtype)
        assert status == 0 and np.array_equal(held, x)
    assert np.array_equal(got[torch.float32], got[torch.bfloat16])
    for t in range(0, T, max(1, T // 300)):
        ref = serve.route_row(x[t], None, k, G, tg, 1, score == "sigmoid", True, 1.0)
        assert np.array_equal(got[torch.float32][t], ref[0]), (t, got[torch.float32][t], ref[0])


@pytest.mark.parametrize("T", [200, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm,offset", [
    ("softmax", True, 60.3), ("softmax", True, 0.7), ("softmax", False, 60.3), ("softmax", False, 0.7),
    ("sigmoid", True, -60.3), ("sigmoid", True, 5.3), ("sigmoid", False, -60.3), ("sigmoid", False, 5.3)])
@pytest.mark.parametrize("E,k", [(128, 8), (1024, 8), (60, 32)])
def test_weights_to_their_last_units(cuda_lib, T, dtype, score, renorm, offset, E, k):
    """The bounds that w4_route states, in units of 2^-24 of a weight: expf 4, a quick quotient 4, a sum,
    a product or a fused one 1 each.  Divided by their sum: softmax terms 5 (an exponential of a
    difference and its rest), their sum 5 + 5 additions, quotient 4, scale 1: 20; sigmoids
    exp / (1 + exp) 5 + 3 + 4, their sum 12 + 5, quotient 4, scale 1: 34.  A sigmoid alone 4 + 1 + 4 + 1:
    10.  A softmax's share 5 + 4 + 1 and the whole sum: at most 63 + 5 additions, and quick exponentials
    4 + 3.4 |d| each, with |d| at most ln(experts) on the average of their weights, 7: 106."""
    rng = np.random.default_rng(E + k + T)
    x = rng.normal(size=(T, E))
    if score == "softmax":
        x[:, rng.integers(0, E)] = offset           # far above the others, or among them
    else:
        x += offset
    ids, w, status, held = run(x, k, 1, 1, 2, score, renorm, 1.5, None, dtype)
    assert status == 0
    units = {("softmax", True): 20, ("sigmoid", True): 34, ("sigmoid", False): 10, ("softmax", False): 106}
    tol = units[score, renorm] * 2.0 ** -24
    for t in range(0, T, max(1, T // 200)):
        ref = serve.route_row(held[t], None, k, 1, 1, 2, score == "sigmoid", renorm, 1.5)
        assert np.array_equal(ids[t], ref[0])
        assert np.all(np.abs(w[t] - ref[1]) <= tol * ref[1] + 1.5 * 2.0 ** -125), \
            (t, np.max(np.abs(w[t] / ref[1] - 1)) * 2.0 ** 24)
