"""Beams that decode through a routed layer and shared pages: every call of a step in turn.

embed_gather -> qkv product -> reserve, append, attention over shared pages -> output product ->
router product, route, routed product, combine -> output table's product -> adjust_logits ->
(tokens and parents drawn on the host) -> fork.  The same steps run once more with a cache of its own
for every beam, copied whole when beams change: the logits have to be the same bits."""

import numpy as np
import pytest
import torch

from bit_weight_only_gemv_gb300 import lib
from oracle import serve

pytestmark = pytest.mark.gpu

HIDDEN, V, E, K = 256, 999, 16, 4
HQ, H, D, P = 8, 2, 64, 16
BEAMS, MAX_PAGES, PROMPT, STEPS = 5, 8, 39, 24


class Model:
    def __init__(self, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def w(n, k, scale=1.0):
            return lib.quantize(torch.randn((n, k), generator=gen, device="cuda") * scale * k ** -0.5)

        self.table = w(V, HIDDEN, 16.0)
        self.qkv, self.o = w((HQ + 2 * H) * D, HIDDEN), w(HIDDEN, HQ * D)
        self.router = w(E, HIDDEN, 2.0)
        self.experts = w(E * HIDDEN, HIDDEN)
        self.bias = 0.05 * torch.randn((E,), generator=gen, device="cuda")
        self.route = lib.Router(E, K, groups=4, top_groups=2, score="sigmoid", scale=1.5)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def product(self, w, x):
        n = lib.workspace_bytes(x.shape[0], w[0].shape[0], x.shape[1])
        ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
        return lib.gemv(*w, x, workspace=ws, status=self.status, pdl=True)

    def routed(self, x):
        """The routed layer of rows x, with its parts."""
        logits = self.product(self.router, x)
        ids, weights = lib.route(self.route, logits, self.bias, self.status)
        qw, st = self.experts
        y = lib.gemv_id(qw, st, ids.view(-1), x.repeat_interleave(K, 0), HIDDEN, HIDDEN, E,
                        HIDDEN * HIDDEN // 2, HIDDEN * HIDDEN // 16, status=self.status, pdl=True)
        out = lib.moe_combine(y, weights, add=x, ids=ids, num_experts=E, status=self.status)
        return out, dict(logits=logits, ids=ids, weights=weights, y=y)

    def layer(self, x, cache, batch):
        rows = self.product(self.qkv, x).view(x.shape[0], HQ + 2 * H, D)
        lib.kv8_append(cache, batch, rows[:, HQ:HQ + H], rows[:, HQ + H:], status=self.status)
        ws = torch.zeros(max(16, lib.kv8_attn_workspace_bytes(cache, batch, HQ, rows=x.shape[0])),
                         dtype=torch.uint8, device="cuda")
        att = lib.kv8_attn(cache, batch, rows[:, :HQ], D ** -0.5, workspace=ws, status=self.status)
        return self.routed(self.product(self.o, att.view(x.shape[0], -1)))


def new_cache(pages):
    return lib.KV8Cache(*(torch.zeros((pages, H, P, D), dtype=torch.uint8, device="cuda") for _ in "kv"),
                        *(torch.zeros((pages, H), device="cuda") for _ in "kv"),
                        ranges=torch.zeros((pages, H, 2, D), dtype=torch.uint8, device="cuda"),
                        weight=torch.zeros((pages, H, P), device="cuda"))


def draws(seed):
    """Tokens of the prompt, and each step's parents (one beam ends now and then)."""
    rng = np.random.default_rng(seed)
    prompt = rng.integers(0, V, PROMPT).astype(np.int32)
    return prompt, [rng.integers(0, BEAMS, BEAMS).astype(np.int32) for _ in range(STEPS)]


def run(shared):
    """Logits of every step; shared: pages by fork and reserve, else a copy of everything."""
    m, (prompt, parents) = Model(), draws(1)
    num = 1 + 3 * BEAMS + MAX_PAGES if shared else BEAMS * MAX_PAGES
    cache = new_cache(num)
    table = torch.full((BEAMS, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros((BEAMS,), dtype=torch.int32, device="cuda")
    refs = torch.zeros((num,), dtype=torch.int32, device="cuda")
    ws = torch.zeros(lib.kv8_pages_workspace_bytes(BEAMS, num), dtype=torch.uint8, device="cuda")
    ids = torch.from_numpy(prompt).cuda()
    x = lib.embed_gather(*m.table, ids, status=m.status)
    grow = torch.tensor([PROMPT] + [0] * (BEAMS - 1), dtype=torch.int32, device="cuda")
    off = torch.tensor([0] + [PROMPT] * BEAMS, dtype=torch.int32, device="cuda")
    if shared:
        lib.kv8_reserve(table, lens, refs, P, grow, ws, m.status)
    else:
        table.copy_(torch.arange(BEAMS * MAX_PAGES, dtype=torch.int32).view(BEAMS, MAX_PAGES))
        lens.copy_(grow)
    m.layer(x, cache, lib.KV8Batch(table, lens, off, rows=PROMPT, max_new=PROMPT, max_len=MAX_PAGES * P))
    first = torch.zeros((BEAMS,), dtype=torch.int32, device="cuda")
    hist = torch.zeros((BEAMS, PROMPT + STEPS), dtype=torch.int32, device="cuda")
    hist[:, :PROMPT] = ids
    count = torch.full((BEAMS,), PROMPT, dtype=torch.int32, device="cuda")
    at = torch.full((BEAMS,), PROMPT, dtype=torch.int32, device="cuda")
    mask = torch.from_numpy(np.random.default_rng(3).integers(-2 ** 31, 2 ** 31, (2, (V + 31) // 32))
                            .astype(np.int32)).cuda()
    rules = lib.LogitRules(tokens=hist, lens=count, prompt=at,
                           repetition=torch.linspace(1.0, 1.4, BEAMS, device="cuda"),
                           presence=torch.full((BEAMS,), 0.3, device="cuda"),
                           frequency=torch.full((BEAMS,), 0.1, device="cuda"), mask=mask,
                           mask_rows=torch.tensor([-1, 0, 1, 0, -1], dtype=torch.int32, device="cuda"))
    out, tokens = [], torch.arange(7, 7 + BEAMS, dtype=torch.int32, device="cuda")
    for step in range(STEPS):
        par = first if step == 0 else torch.from_numpy(parents[step]).cuda()
        if shared:
            table, lens, refs = lib.kv8_fork(cache, table, lens, refs, par, ws, m.status)
            lib.kv8_reserve(table, lens, refs, P, None, ws, m.status)
            if step % 7 == 6:
                table, refs, _ = lib.kv8_compact(cache, table, lens, refs, ws, m.status)
        else:
            for t in cache.tensors:
                rows = t.view(BEAMS, MAX_PAGES, *t.shape[1:])
                rows.copy_(rows[par.long()].clone())
            lens = lens[par.long()] + 1
        hist.copy_(hist[par.long()].clone())
        tokens = tokens[par.long()]
        hist[torch.arange(BEAMS), count.long()] = tokens
        count += 1
        x = lib.embed_gather(*m.table, tokens, status=m.status)
        batch = lib.KV8Batch(table, lens, max_len=MAX_PAGES * P)
        h, parts = m.layer(x, cache, batch)
        logits = m.product(m.table, h)
        raw = logits.clone()
        lib.adjust_logits(logits, rules, m.status)
        # beams of one parent take different tokens: the best, the second best, ...
        best = logits.float().topk(BEAMS, dim=1).indices.to(torch.int32)
        tokens = best[torch.arange(BEAMS), torch.arange(BEAMS)].contiguous()
        out.append(dict(raw=raw.clone(), adjusted=logits.clone(), hist=hist.clone(), count=count.clone(),
                        h=h.clone(), **{k: v.clone() for k, v in parts.items()}))
        assert int(m.status) == 0
    if shared:      # every page is counted as often as it is named
        named = torch.zeros_like(refs)
        for b in range(BEAMS):
            for p in table[b, :-(-int(lens[b]) // P)].tolist():
                named[p] += 1
        assert torch.equal(named, refs)
        assert int((refs > 1).sum()) > 0
    return out, m, rules


def test_shared_pages_give_the_bits_of_caches_of_their_own(cuda_lib):
    a, b = run(True)[0], run(False)[0]
    for step, (x, y) in enumerate(zip(a, b)):
        for k in x:
            assert torch.equal(x[k], y[k]), (step, k)


def test_each_step_against_the_references(cuda_lib):
    out, m, rules = run(True)
    bias = m.bias.double().cpu().numpy()
    r = {k: t.cpu().numpy() for k, t in zip(("rep", "pres", "freq"), rules.tensors[3:6])}
    mask = np.unpackbits(rules.tensors[9].cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :V]
    rows = rules.tensors[10].tolist()
    for s in out[::5]:
        x = s["logits"].double().cpu().numpy()
        for b in range(BEAMS):
            ids, w = serve.route_row(x[b], bias, K, 4, 2, 2, True, True, 1.5)
            assert np.array_equal(s["ids"][b].cpu().numpy(), ids)
            assert np.allclose(s["weights"][b].cpu().numpy(), w, rtol=2.0 ** -18, atol=0)
    for s in out[::5]:
        raw, got = s["raw"].double().cpu().numpy(), s["adjusted"].double().cpu().numpy()
        for b in range(BEAMS):
            ref, size, _ = serve.adjust_row(raw[b], s["hist"][b, :int(s["count"][b])].tolist(), PROMPT,
                                            float(r["rep"][b]), float(r["pres"][b]), float(r["freq"][b]),
                                            mask=None if rows[b] < 0 else mask[rows[b]].astype(bool))
            with np.errstate(invalid="ignore"):
                near = np.abs(got[b] - ref) <= 5 * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(ref)
            ok = (got[b] == ref) | near
            assert ok.all()


def test_a_routed_step_in_a_graph(cuda_lib):
    """Route, the experts' products, their sum and the logits' rules captured once, replayed on other
    inputs: the bits of the calls one by one."""
    m = Model(5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((BEAMS, HIDDEN), generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.empty((BEAMS, K), dtype=torch.int32, device="cuda")
    weights = torch.empty((BEAMS, K), device="cuda")
    logits = torch.empty((BEAMS, E), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((BEAMS * K, HIDDEN), dtype=torch.bfloat16, device="cuda")
    xs = torch.empty((BEAMS * K, HIDDEN), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((BEAMS, HIDDEN), dtype=torch.bfloat16, device="cuda")
    head = torch.empty((BEAMS, V), dtype=torch.bfloat16, device="cuda")
    hist = torch.randint(0, V, (BEAMS, 50), generator=gen, device="cuda", dtype=torch.int32)
    rules = lib.LogitRules(tokens=hist, lens=torch.full((BEAMS,), 50, dtype=torch.int32, device="cuda"),
                           repetition=torch.full((BEAMS,), 1.2, device="cuda"))
    n = max(lib.workspace_bytes(BEAMS, k, HIDDEN) for k in (E, V))
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    qw, st = m.experts

    def step():
        lib.gemv(*m.router, x, y=logits, workspace=ws, status=m.status, pdl=True)
        lib.bind_route(m.route, logits, ids, weights, m.bias, m.status)()
        xs.copy_(x.repeat_interleave(K, 0))
        lib.gemv_id(qw, st, ids.view(-1), xs, HIDDEN, HIDDEN, E, HIDDEN * HIDDEN // 2,
                    HIDDEN * HIDDEN // 16, y=y, status=m.status, pdl=True)
        lib.moe_combine(y, weights, out, x, ids, E, m.status)
        lib.gemv(*m.table, out, y=head, workspace=ws, status=m.status, pdl=True)
        lib.adjust_logits(head, rules, m.status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda").to(torch.bfloat16))
        g.replay()
        got = [t.clone() for t in (ids, weights, out, head)]
        for t in (ids, weights, out, head):
            t.zero_()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (ids, weights, out, head)))
    assert int(m.status) == 0


def test_calls_on_another_stream(cuda_lib):
    """Inputs made on one stream, the call and its fresh outputs on another."""
    m = Model(7)
    side = torch.cuda.Stream()
    x = torch.randn((300, E), device="cuda")
    want = lib.route(m.route, x, m.bias)
    torch.cuda.synchronize()
    for _ in range(20):
        z = torch.empty_like(x).copy_(x)
        side.wait_stream(torch.cuda.current_stream())
        got = lib.route(m.route, z, m.bias, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_one_workspace_for_every_call(cuda_lib):
    """A split-K product, attention and the page calls on one buffer, in turn: the results of buffers
    of their own."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    w = lib.quantize(torch.randn((16, 21504), generator=gen, device="cuda") * 0.01)
    x = torch.randn((1, 21504), generator=gen, device="cuda").to(torch.bfloat16)
    cache = new_cache(40)
    for t in cache.tensors[:2]:
        t.random_(0, 256, generator=gen)
    for t in cache.tensors[2:4]:
        t.fill_(2.0 ** -7)
    table = torch.randperm(40, generator=gen, device="cuda")[:16].to(torch.int32).view(2, 8).contiguous()
    lens = torch.tensor([120, 87], dtype=torch.int32, device="cuda")
    refs = torch.zeros((40,), dtype=torch.int32, device="cuda")
    refs[table[0].long()] = 1
    refs[table[1, :6].long()] = 1
    q = torch.randn((2, HQ, D), generator=gen, device="cuda").to(torch.bfloat16)
    batch = lib.KV8Batch(table, lens, max_len=128)
    parents = torch.tensor([1, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
    sizes = [lib.workspace_bytes(1, 16, 21504), lib.kv8_attn_workspace_bytes(cache, batch, HQ),
             lib.kv8_pages_workspace_bytes(5, 40)]
    assert all(sizes)
    one = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")

    def calls(ws):
        got = [lib.gemv(*w, x, workspace=ws(0)), lib.kv8_attn(cache, batch, q, 0.125, workspace=ws(1))]
        t, n, r = lib.kv8_fork(cache, table, lens, refs, parents, ws(2))
        lib.kv8_reserve(t, n, r, P, None, ws(2))
        got += [t, n, r, *lib.kv8_compact(cache, t, n, r, ws(2))]
        return [g.clone() for g in got]

    want = calls(lambda i: torch.zeros(sizes[i], dtype=torch.uint8, device="cuda"))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, calls(lambda i: one)))


def test_two_streams_at_once(cuda_lib):
    """The same calls on buffers of their own, on two streams at the same time: the results of each alone."""
    from _pages import Pages
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sides = []
    for i in range(2):
        p = Pages(20 + i, [300, 41, 77, 16], layers=6, spare=30).to_gpu(most_rows=8)
        gen = torch.Generator(device="cuda").manual_seed(i)
        sides.append(dict(p=p, parents=torch.tensor([0, 0, 1, 2, 3, 0], dtype=torch.int32, device="cuda"),
                          x=torch.randn((700, 64), generator=gen, device="cuda"),
                          head=torch.randn((9, 5001), generator=gen, device="cuda"),
                          hist=torch.randint(0, 5001, (9, 800), generator=gen, device="cuda", dtype=torch.int32)))

    def calls(s, stream):
        p = s["p"]
        ids, w = lib.route(lib.Router(64, 5, groups=8, top_groups=3, score="sigmoid"), s["x"], stream=stream)
        head = s["head"].clone()
        rules = lib.LogitRules(tokens=s["hist"], lens=torch.full((9,), 800, dtype=torch.int32, device="cuda"),
                               frequency=torch.full((9,), 0.25, device="cuda"))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        lib.adjust_logits(head, rules, p.status, stream=stream)
        t, n, r = lib.kv8_fork(p.dev, p.table, p.lens, p.refs, s["parents"], p.ws, p.status, stream=stream)
        lib.kv8_reserve(t, n, r, p.P, None, p.ws, p.status, stream=stream)
        return [ids, w, head, t, n, r, rules]

    alone = []
    for s in sides:
        alone.append(calls(s, None)[:-1])
        torch.cuda.synchronize()
    for _ in range(25):
        both = [calls(s, stream) for s, stream in zip(sides, streams)]
        torch.cuda.synchronize()
        for one, two in zip(alone, both):
            assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert all(int(s["p"].status) == 0 for s in sides)
