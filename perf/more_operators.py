"""Operators between the products of a decode step: plain forms, the library's calls, and the cases that time them.

A batch that decodes through routed layers and a paged cache needs, besides the
4-bit products and the attention:

route    which experts a token goes to, and with what weights, from the router's logits
combine  the chosen experts' output rows added up by those weights
logits   the output product's logits with penalties for repeated tokens, biases and a
         grammar's mask, in place
fork     sequences that continue others (or end): their pages shared, the page that a
         sequence will write to its own copy, the pages of nobody free again; then a page
         for each next token that needs one
compact  the pages in use moved to the lowest numbers

The formulas:

route    s = softmax(logits) or sigmoid(logits); c = s + bias; a group's score is the sum of
         its one or two largest c; the top_k experts of largest c within the best top_groups
         groups, in order of c, equal ones from the lowest number on; weights scale * s, or
         scale * s / (sum of the chosen s)
combine  out[t] = add[t] + sum_j weights[t][j] * y[t * top_k + j]
logits   x > 0 ? x / repetition : x * repetition where the token occurs in the row's history;
         - frequency * n - presence (n > 0) for its n occurrences after the prompt; + bias;
         -inf where the mask's bit is 0
"""

import math

import torch

own = False

_DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # batch-1 decode through a routed layer: 128 experts, top 8 (the 30-layer hidden-2816 decoder)
        dict(name="route-token", op="route", T=1, E=128, k=8, groups=1, top_groups=1, best=1,
             score="softmax", bias=False, renorm=True, dtype="bf16"),
        # a serving batch of 192 sequences, sigmoid scores with balancing biases and groups
        dict(name="route-batch", op="route", T=192, E=256, k=8, groups=8, top_groups=4, best=2,
             score="sigmoid", bias=True, renorm=True, dtype="fp32"),
        # sixty-four prompt chunks of 256 tokens
        dict(name="route-chunks", op="route", T=16384, E=256, k=8, groups=8, top_groups=4, best=2,
             score="sigmoid", bias=True, renorm=True, dtype="bf16"),
        # one token's eight expert rows of the hidden-2816 decoder
        dict(name="combine-token", op="combine", T=1, k=8, N=2816, add=False),
        # a ragged batch of prompts, with the dense branch's output added
        dict(name="combine-chunks", op="combine", T=4001, k=8, N=2816, add=True),
        # batch-1 decode over the 262144-token vocabulary, penalties only
        dict(name="logits-token", op="logits", B=1, V=262144, L=700, dtype="bf16", nb=0, mask=False),
        # 24 conversations, most of them under a grammar, 300 biased tokens each
        dict(name="logits-grammar", op="logits", B=24, V=262144, L=4096, dtype="bf16", nb=300,
             mask=True),
        # 64 long conversations over a smaller vocabulary of odd size, logits in 32 bits
        dict(name="logits-batch", op="logits", B=64, V=100277, L=30000, dtype="fp32", nb=64,
             mask=True),
        # four beams of one conversation, two layers
        dict(name="fork-beams", op="fork", C=1, W=4, L=700, tail=90, layers=2, H=2, D=256, P=16),
        # a step of eight beams in each of sixteen conversations, thirty layers
        dict(name="fork-batch", op="fork", C=16, W=8, L=2000, tail=120, layers=30, H=8, D=128, P=32),
        # a small pool after half of its sequences have ended
        dict(name="compact-small", op="compact", B=6, L=500, live=0.5, layers=4, H=2, D=256, P=16),
        # a pool of 3400 pages in sixteen layers, about a third of them in use
        dict(name="compact-pool", op="compact", B=40, L=1800, live=0.33, layers=16, H=4, D=128, P=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "combine", "logits", "logits", "fork", "compact"])
    if op == "route":
        E = rng.choice([4, 8, 16, 24, 60, 64, 96, 128, 128, 160, 256, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        top_groups = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 4, 6, 8, 8, 10, 16]), top_groups * (E // groups))
        c = dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, groups=groups, top_groups=top_groups,
                 best=rng.choice([1, 2]), score=rng.choice(["softmax", "sigmoid"]),
                 bias=rng.random() < 0.5, renorm=rng.random() < 0.7,
                 dtype=rng.choice(["bf16", "fp32"]))
        while c["T"] * E > 2 ** 22:
            c["T"] = c["T"] * 3 // 4
        return c
    if op == "combine":
        c = dict(op=op, T=_log(rng, 1, 8192), k=rng.choice([1, 2, 4, 6, 8, 8, 11, 16]),
                 N=_log(rng, 65, 8192), add=rng.random() < 0.5)
        if rng.random() < 0.7:
            c["N"] = (c["N"] + 31) // 32 * 32
        while c["T"] * c["k"] * c["N"] > 4001 * 8 * 2816:
            c["T"] = c["T"] * 3 // 4
        return c
    if op == "logits":
        c = dict(op=op, B=_log(rng, 1, 64), V=_log(rng, 1000, 262144), L=_log(rng, 1, 30000),
                 dtype=rng.choice(["bf16", "bf16", "fp32"]), nb=rng.choice([0, 7, 64, 300, 1000]),
                 mask=rng.random() < 0.6)
        while c["B"] * c["V"] > 24 * 262144:
            c["B"] = max(1, c["B"] * 3 // 4)
        return c
    D, P, H = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    if op == "fork":
        c = dict(op=op, C=_log(rng, 1, 16), W=rng.choice([1, 2, 3, 4, 8, 16]), L=_log(rng, 2, 8000),
                 layers=_log(rng, 1, 32), H=H, D=D, P=P)
        c["tail"] = _log(rng, 1, 300)
        while c["C"] * (c["L"] + (c["W"] + 1) * (c["tail"] + 2 * P)) * c["layers"] * H * D > 2 ** 30:
            c["C"], c["layers"] = max(1, c["C"] * 3 // 4), max(1, c["layers"] * 3 // 4)
            c["L"] = max(2, c["L"] * 3 // 4)
        return c
    c = dict(op=op, B=_log(rng, 1, 48), L=_log(rng, 20, 4000), live=round(rng.uniform(0.2, 0.95), 2),
             layers=_log(rng, 1, 16), H=H, D=D, P=P)
    while c["B"] * (c["L"] + P) * c["layers"] * H * D / c["live"] > 2 ** 30:
        c["B"], c["layers"] = max(1, c["B"] * 3 // 4), max(1, c["layers"] * 3 // 4)
        c["L"] = max(20, c["L"] * 3 // 4)
    return c


def _histories(c):
    """Tokens so far of each row: the first has L, the others L/4 to L."""
    L = c["L"]
    return [L if b == 0 else L - (3 * L * (29 * b % 53)) // (4 * 53) for b in range(c["B"])]


def _mask_of(c, b):
    """Share of the vocabulary that row b's grammar allows (None: no grammar): a keyword or a
    number, the inside of a string, free text."""
    return (None, 0.002, 0.95, 0.02)[b % 4] if c["mask"] and c["B"] > 1 else 0.01 if c["mask"] else None


def _conversations(c):
    """Lengths of the conversations of a fork: the first has L, the others L/2 to L."""
    L = c["L"]
    return [L if i == 0 else max(2, L - (L * (17 * i % 31)) // (2 * 31)) for i in range(c["C"])]


def _page_bytes(c, tokens):
    """Bytes of one page in one layer of which `tokens` are in use: codes, steps, ranges, weights."""
    return c["H"] * (2 * tokens * c["D"] + 8 + 2 * c["D"] + 4 * tokens)


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    c, op = case, case["op"]
    if op == "route":
        n, el = c["T"] * c["E"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": n * el + c["E"] * 4 * c["bias"] + c["T"] * c["k"] * 8, "flops": 4 * n}
    if op == "combine":
        n = c["T"] * c["N"]
        return {"bytes": 2 * n * (c["k"] + 1 + c["add"]) + c["T"] * c["k"] * 8, "flops": 2 * n * c["k"]}
    if op == "logits":
        el, nbytes = 2 if c["dtype"] == "bf16" else 4, 0
        for b, n in enumerate(_histories(c)):
            share = _mask_of(c, b)
            touched = min(c["V"], n // 2 + c["nb"])      # a history names about half as many tokens
            nbytes += 4 * n + 8 * c["nb"] + 12
            if share is None:
                nbytes += 2 * touched * el
            else:                                        # the mask, -inf where it says no, the rest
                nbytes += c["V"] // 8 + int(c["V"] * (1 - share)) * el + int(2 * touched * share) * el
        return {"bytes": nbytes, "flops": 0}
    P = c["P"]
    if op == "fork":
        lens = _conversations(c)
        entries = sum(c["W"] * -(-n // P) for n in lens)
        # of W draws from W rows about W / e are repeated: each copies the page in use
        copied = [(c["W"] - c["W"] * (1 - (1 - 1 / c["W"]) ** c["W"])) * _page_bytes(c, n % P)
                  for n in lens if n % P]
        return {"bytes": 8 * entries + 2 * int(sum(copied)) * c["layers"], "flops": 0}
    pages = sum(-(-n // P) for n in _histories(c))
    moved = int(pages * (1 - c["live"]))
    return {"bytes": 8 * pages + 2 * moved * c["layers"] * _page_bytes(c, P), "flops": 0}


# ------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _pool(s, gen, num):
    """Random codes, steps, ranges and weights of `num` pages in every layer."""
    c = s["case"]
    n, H, P, D = c["layers"], c["H"], c["P"], c["D"]
    for k in ("kc", "vc"):
        s[k] = torch.randint(0, 256, (n, num, H, P, D), generator=gen, device=_DEV, dtype=torch.uint8)
    for k in ("ks", "vs"):
        e = torch.randint(-12, -4, (n, num, H), generator=gen, device=_DEV)
        s[k] = torch.exp2(e.float())
    s["ranges"] = torch.stack([s["kc"].amin(3), s["kc"].amax(3)], 3)
    s["weight"] = torch.rand((n, num, H, P), generator=gen, device=_DEV)


def _prepare_route(c, s, gen):
    x = torch.randn((c["T"], c["E"]), generator=gen, device=_DEV) * 1.3
    x = x + 0.7 * torch.randn((1, c["E"]), generator=gen, device=_DEV)      # some experts are liked
    s["logits"] = x.to(_TYPES[c["dtype"]])
    s["bias"] = 0.05 * torch.randn((c["E"],), generator=gen, device=_DEV) if c["bias"] else None
    s["ids"] = torch.empty((c["T"], c["k"]), dtype=torch.int32, device=_DEV)
    s["weights"] = torch.empty((c["T"], c["k"]), dtype=torch.float32, device=_DEV)


def _prepare_combine(c, s, gen):
    T, k, N = c["T"], c["k"], c["N"]
    s["y"] = torch.randn((T * k, N), generator=gen, device=_DEV).to(torch.bfloat16)
    w = torch.rand((T, k), generator=gen, device=_DEV) + 0.05
    s["weights"] = (w / w.sum(1, keepdim=True)).contiguous()
    s["ids"] = torch.randint(0, 128, (T, k), generator=gen, device=_DEV, dtype=torch.int32)
    s["add"] = torch.randn((T, N), generator=gen, device=_DEV).to(torch.bfloat16) if c["add"] else None
    s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device=_DEV)


def _prepare_logits(c, s, gen):
    B, V, lens = c["B"], c["V"], _histories(c)
    s["logits"] = (3 * torch.randn((B, V), generator=gen, device=_DEV)).to(_TYPES[c["dtype"]])
    # few tokens often, most of them seldom
    u = torch.rand((B, c["L"]), generator=gen, device=_DEV, dtype=torch.float64)
    s["tokens"] = (V * u ** 4).to(torch.int32).clamp(max=V - 1)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_DEV)
    s["prompt"] = torch.tensor([n * (b % 3) // 3 for b, n in enumerate(lens)], dtype=torch.int32,
                               device=_DEV)
    for name, lo, hi in (("repetition", 1.0, 1.3), ("presence", 0.0, 0.6), ("frequency", 0.0, 0.2)):
        s[name] = lo + (hi - lo) * torch.rand((B,), generator=gen, device=_DEV)
    s["bias_ids"] = s["bias"] = s["n_bias"] = None
    if c["nb"]:
        nb = min(c["nb"], V)
        key = torch.rand((B, V), generator=gen, device=_DEV)
        s["bias_ids"] = key.topk(nb).indices.to(torch.int32)
        s["bias"] = 4 * torch.randn((B, nb), generator=gen, device=_DEV)
        s["n_bias"] = torch.tensor([nb if b % 3 else nb // 2 for b in range(B)], dtype=torch.int32,
                                   device=_DEV)
    s["mask"] = s["mask_rows"] = None
    if c["mask"]:
        shares = [_mask_of(c, b) for b in range(B)]
        with_mask = [i for i, x in enumerate(shares) if x is not None]
        share = torch.tensor([shares[i] for i in with_mask], device=_DEV)
        words = -(-V // 32)
        bits = torch.rand((len(with_mask), words, 32), generator=gen, device=_DEV) < share[:, None, None]
        w = (bits.long() << torch.arange(32, device=_DEV)).sum(-1)
        s["mask"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
        at = {b: i for i, b in enumerate(with_mask)}
        s["mask_rows"] = torch.tensor([at.get(b, -1) for b in range(B)], dtype=torch.int32, device=_DEV)


def _tables(s, gen, rows, num):
    """Page table of rows given as lists of page names, on pages drawn from `num`; references."""
    order = torch.randperm(num, generator=gen, device=_DEV).tolist()
    mp = max(len(r) for r in rows) + 1
    names = {}
    full = [[order[names.setdefault(p, len(names))] for p in r] + [-1] * (mp - len(r)) for r in rows]
    s["table"] = torch.tensor(full, dtype=torch.int32, device=_DEV)
    refs = [0] * num
    for r in full:
        for p in r:
            if p >= 0:
                refs[p] += 1
    s["refs"] = torch.tensor(refs, dtype=torch.int32, device=_DEV)
    s["num"] = num


def _prepare_fork(c, s, gen):
    P, rows, lens = c["P"], [], []
    for i, n in enumerate(_conversations(c)):
        pages = -(-n // P)
        shared = max(0, n - c["tail"]) // P
        for w in range(c["W"]):
            rows.append([(i, -1, p) if p < shared else (i, w, p) for p in range(pages)])
            lens.append(n)
    used = len({p for r in rows for p in r})
    B = len(rows)
    num = used + 2 * B + 3
    _pool(s, gen, num)
    _tables(s, gen, rows, num)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_DEV)
    pick = torch.randint(0, c["W"], (c["C"], c["W"]), generator=gen, device=_DEV)
    par = (pick + c["W"] * torch.arange(c["C"], device=_DEV)[:, None]).to(torch.int32)
    if c["C"] > 2:
        par[-1] = -1                                    # one conversation has ended
    s["parents"] = par.view(-1).contiguous()
    s["new_table"] = torch.full_like(s["table"], -1)
    s["new_lens"] = torch.zeros_like(s["lens"])
    s["new_refs"] = torch.zeros_like(s["refs"])


def _prepare_compact(c, s, gen):
    P, lens = c["P"], _histories(c)
    # every other row continues the one before it: half of its pages are that row's
    rows = []
    for b, n in enumerate(lens):
        pages = -(-n // P)
        common = min(pages, lens[b - 1] // P) // 2 if b % 2 else 0
        rows.append([(b - 1, p) if p < common else (b, p) for p in range(pages)])
    used = len({p for r in rows for p in r})
    num = max(used + 1, int(used / c["live"]))
    _pool(s, gen, num)
    _tables(s, gen, rows, num)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_DEV)
    s["new_table"] = torch.full_like(s["table"], -1)
    s["new_refs"] = torch.zeros_like(s["refs"])
    s["used"] = torch.zeros((1,), dtype=torch.int32, device=_DEV)


_PREPARE = {"route": _prepare_route, "combine": _prepare_combine, "logits": _prepare_logits,
            "fork": _prepare_fork, "compact": _prepare_compact}


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    s = dict(case=case)
    _PREPARE[case["op"]](case, s, gen)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].double()             # scores next to a border: in 64 bits
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score if s["bias"] is None else score + s["bias"].double()
    rank = x if s["bias"] is None else choice      # the scores' order is the logits'
    if G > 1:
        each = choice.view(T, G, E // G)
        best = torch.sort(each, dim=-1, descending=True).values[..., :c["best"]].sum(-1)
        if s["bias"] is None and c["best"] == 1:
            best = x.view(T, G, E // G).amax(-1)
        order = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        inside = torch.zeros((T, G), dtype=torch.bool, device=_DEV).scatter_(1, order, True)
        rank = torch.where(inside.repeat_interleave(E // G, 1), rank, -math.inf)
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    s["ids"], s["weights"] = ids.to(torch.int32), (_SCALE * w).float()
    return {"ids": s["ids"], "weights": s["weights"]}


_SCALE = 1.5


def _plain_combine(s):
    c = s["case"]
    y = s["y"].float().view(c["T"], c["k"], c["N"])
    out = (s["weights"][..., None] * y).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    s["out"] = out.to(torch.bfloat16)
    return {"out": s["out"]}


def _plain_logits(s):
    c = s["case"]
    B, V = c["B"], c["V"]
    at = torch.arange(c["L"], device=_DEV)[None]
    live = at < s["lens"][:, None]
    after = live & (at >= s["prompt"][:, None])
    tok = s["tokens"].long()
    n = torch.zeros((B, V), device=_DEV).scatter_add_(1, tok, after.float())
    seen = torch.zeros((B, V), device=_DEV).scatter_add_(1, tok, live.float()) > 0
    x = s["logits"].float()
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * n - s["presence"][:, None] * (n > 0)
    if s["bias"] is not None:
        real = torch.arange(s["bias"].shape[1], device=_DEV)[None] < s["n_bias"][:, None]
        x = x.scatter_add(1, s["bias_ids"].long(), torch.where(real, s["bias"], 0.0))
    if s["mask"] is not None:
        words = s["mask"][s["mask_rows"].clamp(min=0).long()]
        bits = (words[..., None] >> torch.arange(32, device=_DEV)) & 1
        ok = bits.flatten(1)[:, :V].bool() | (s["mask_rows"] < 0)[:, None]
        x = torch.where(ok, x, -math.inf)
    s["logits"].copy_(x)
    return {"logits": s["logits"]}


def _count(num, pages, valid):
    """How often each page is named."""
    n = torch.zeros(num + 1, dtype=torch.int32, device=_DEV)
    at = torch.where(valid, pages, num).flatten().long()
    return n.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:num]


def _move(s, src, dst, tokens):
    """Pages src to dst, the first `tokens` tokens of each, in every layer."""
    some = torch.arange(s["case"]["P"], device=_DEV)[None] < tokens[:, None]           # [n, P]
    for_codes, for_weight = some[None, :, None, :, None], some[None, :, None, :]
    s["kc"][:, dst] = torch.where(for_codes, s["kc"][:, src], s["kc"][:, dst])
    s["vc"][:, dst] = torch.where(for_codes, s["vc"][:, src], s["vc"][:, dst])
    s["weight"][:, dst] = torch.where(for_weight, s["weight"][:, src], s["weight"][:, dst])
    s["ks"][:, dst] = s["ks"][:, src]
    s["vs"][:, dst] = s["vs"][:, src]
    s["ranges"][:, dst] = s["ranges"][:, src]


def _plain_fork(s):
    P, num, old = s["case"]["P"], s["num"], s["table"]
    B, mp = old.shape
    at, row = torch.arange(mp, device=_DEV)[None], torch.arange(B, device=_DEV)
    par = s["parents"].clamp(min=0).long()
    lens = torch.where(s["parents"] >= 0, s["lens"][par], 0)
    pages, had = (lens + P - 1) // P, (s["lens"] + P - 1) // P
    valid = at < pages[:, None]
    table = torch.where(valid, old[par], s["new_table"])
    refs = s["refs"] - _count(num, old, at < had[:, None]) + _count(num, table, valid)
    # the page that a row will write to: its own, or the first row's of those that end in it
    last = table.gather(1, (pages - 1).clamp(min=0).long()[:, None])[:, 0]
    open_ = lens % P > 0
    ends = _count(num, last, open_)
    q = torch.where(open_, last, num).long()
    first = torch.full((num + 1,), B, device=_DEV).scatter_reduce_(0, q, row, "amin")
    refs_of = refs[q.clamp(max=num - 1)]
    copy = open_ & ~((ends[q.clamp(max=num - 1)] == refs_of) & (first[q] == row))
    free = (refs == 0).nonzero()[:, 0]
    dst = free[(torch.cumsum(copy, 0) - 1).clamp(min=0)]
    src, to, rows = q[copy], dst[copy], row[copy]
    _move(s, src, to, (lens % P)[copy])
    table[rows, (pages[copy] - 1).long()] = to.to(torch.int32)
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    refs[to] = 1
    # the next token of each row that goes on: a page where the last one is full
    more = (lens > 0) & (lens % P == 0)
    free = (refs == 0).nonzero()[:, 0]
    dst = free[(torch.cumsum(more, 0) - 1).clamp(min=0)]
    table[row[more], pages[more].long()] = dst[more].to(torch.int32)
    refs[dst[more]] = 1
    s["new_table"], s["new_refs"] = table, refs
    s["new_lens"] = (lens + (lens > 0)).to(torch.int32)
    return {k: s[k] for k in _GIVES["fork"]}


def _plain_compact(s):
    P, num, old = s["case"]["P"], s["num"], s["table"]
    at = torch.arange(old.shape[1], device=_DEV)[None]
    valid = at < ((s["lens"] + P - 1) // P)[:, None]
    page, live = torch.arange(num, device=_DEV), s["refs"] != 0
    n = live.sum()
    src = (live & (_count(num, old, valid) == s["refs"]) & (page >= n)).nonzero()[:, 0]
    dst = (~live & (page < n)).nonzero()[:, 0][:src.numel()]
    _move(s, src, dst, torch.full_like(src, P))
    to = page.clone()
    to[src] = dst
    refs = s["refs"].clone()
    refs[dst] = refs[src]
    refs[src] = 0
    s["new_table"] = torch.where(valid, to[old.clamp(min=0).long()].to(torch.int32), s["new_table"])
    s["new_refs"] = refs
    s["used"] = torch.where(refs != 0, page + 1, 0).amax().view(1).to(torch.int32)
    return {k: s[k] for k in _GIVES["compact"]}


_PLAIN = {"route": _plain_route, "combine": _plain_combine, "logits": _plain_logits,
          "fork": _plain_fork, "compact": _plain_compact}

_POOL = ("kc", "vc", "ks", "vs", "ranges", "weight")
_GIVES = {"route": ("ids", "weights"), "combine": ("out",), "logits": ("logits",),
          "fork": ("new_table", "new_lens", "new_refs", *_POOL),
          "compact": ("new_table", "new_refs", "used", *_POOL)}


# ------------------------------------------------------------------ the library's calls
def _bound(s):
    """The calls of a serving loop on these buffers, marshalled once, as such a loop keeps them."""
    from bit_weight_only_gemv_gb300 import lib

    c, op = s["case"], s["case"]["op"]
    if op == "route":
        router = lib.Router(c["E"], c["k"], groups=c["groups"], top_groups=c["top_groups"],
                            group_best=c["best"], score=c["score"], renorm=c["renorm"], scale=_SCALE)
        return [lib.bind_route(router, s["logits"], s["ids"], s["weights"], bias=s["bias"])]
    if op == "combine":
        return [lib.bind_moe_combine(s["y"], s["weights"], s["out"], add=s["add"], ids=s["ids"],
                                     num_experts=128)]
    if op == "logits":
        rules = lib.LogitRules(tokens=s["tokens"], lens=s["lens"], prompt=s["prompt"],
                               repetition=s["repetition"], presence=s["presence"],
                               frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                               n_bias=s["n_bias"], mask=s["mask"], mask_rows=s["mask_rows"])
        return [lib.bind_adjust_logits(s["logits"], rules)]
    caches = [lib.KV8Cache(*(s[k][i] for k in _POOL)) for i in range(c["layers"])]
    need = lib.kv8_pages_workspace_bytes(s["table"].shape[0], s["num"])
    ws = torch.zeros(need, dtype=torch.uint8, device=_DEV)
    if op == "fork":
        return [lib.bind_kv8_fork(caches, s["table"], s["lens"], s["refs"], s["parents"],
                                  s["new_table"], s["new_lens"], s["new_refs"], workspace=ws),
                lib.bind_kv8_reserve(s["new_table"], s["new_lens"], s["new_refs"], c["P"],
                                     workspace=ws)]
    return [lib.bind_kv8_compact(caches, s["table"], s["lens"], s["refs"], s["new_table"],
                                 s["new_refs"], s["used"], workspace=ws)]


def run(state):
    op = state["case"]["op"]
    if not own:
        return _PLAIN[op](state)
    if "calls" not in state:
        state["calls"] = _bound(state)
    for call in state["calls"]:
        call()
    return {k: state[k] for k in _GIVES[op]}


# ------------------------------------------------------------------ definition in 64 bits
def _exact_route(c, s):
    x = s["logits"].double()
    score = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    choice = score + (s["bias"].double() if s["bias"] is not None else 0.0)
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        best = choice.unflatten(1, (c["groups"], size)).topk(min(c["best"], size), 2).values.sum(2)
        out = torch.ones_like(best, dtype=torch.bool)
        out.scatter_(1, best.topk(c["top_groups"], 1).indices, False)
        choice = choice.masked_fill(out.repeat_interleave(size, 1), -math.inf)
    w = torch.gather(score, 1, choice.topk(c["k"], 1).indices)
    return {"ids": None, "weights": _SCALE * (w / w.sum(1, keepdim=True) if c["renorm"] else w)}


def _exact_logits(c, s):
    out = s["logits"].double()
    lens, prompt = s["lens"].tolist(), s["prompt"].tolist()
    for b in range(c["B"]):
        row, hist = out[b], s["tokens"][b, :lens[b]].long()
        n = torch.bincount(hist[prompt[b]:], minlength=c["V"]).double()
        seen = torch.unique(hist)
        r = float(s["repetition"][b])
        row[seen] = torch.where(row[seen] > 0, row[seen] / r, row[seen] * r)
        row -= float(s["frequency"][b]) * n + float(s["presence"][b]) * n.clamp(max=1)
        if s["bias"] is not None:
            m = int(s["n_bias"][b])
            row[s["bias_ids"][b, :m].long()] += s["bias"][b, :m].double()
        g = -1 if s["mask"] is None else int(s["mask_rows"][b])
        if g >= 0:
            v = torch.arange(c["V"], device=_DEV)
            row[(s["mask"][g][v // 32] >> (v % 32)) % 2 == 0] = -math.inf
    return {"logits": out}


def _exact_pages(c, s):
    """Steps and weights after the copies, page by page (codes, tables and counts have no value but
    the stored one)."""
    P, refs, lens = c["P"], s["refs"].tolist(), s["lens"].tolist()
    table = s["table"].tolist()
    copies = []
    if c["op"] == "fork":
        after = list(refs)
        rows, ends = [], {}
        for b, p in enumerate(s["parents"].tolist()):
            for q in table[b][:-(-lens[b] // P)]:
                after[q] -= 1
            rows.append(table[p][:-(-lens[p] // P)] if p >= 0 else [])
            for q in rows[-1]:
                after[q] += 1
            if rows[-1] and lens[p] % P:
                ends.setdefault(rows[-1][-1], []).append((b, lens[p] % P))
        free = iter([q for q, n in enumerate(after) if n == 0])
        todo = []
        for q, who in ends.items():
            todo += [(b, q, n) for b, n in (who[1:] if len(who) == after[q] else who)]
        copies = [(q, next(free), n) for _, q, n in sorted(todo)]
    else:
        live = [q for q, n in enumerate(refs) if n]
        holes = iter([q for q, n in enumerate(refs[:len(live)]) if not n])
        copies = [(q, next(holes), P) for q in live if q >= len(live)]
    got = {k: s[k].double() for k in ("ks", "vs", "weight")}
    if copies:
        src, dst, n = torch.tensor(copies, device=_DEV).T
        got["ks"][:, dst], got["vs"][:, dst] = got["ks"][:, src], got["vs"][:, src]
        lo = torch.arange(P, device=_DEV) < n[:, None]
        i, t = lo.nonzero().T
        got["weight"][:, dst[i], :, t] = got["weight"][:, src[i], :, t]
    return {k: got.get(k) for k in _GIVES[c["op"]]}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "combine":
        y = s["y"].double().unflatten(0, (case["T"], case["k"]))
        out = torch.einsum("tk,tkn->tn", s["weights"].double(), y)
        return {"out": out if s["add"] is None else out + s["add"].double()}
    if op == "logits":
        return _exact_logits(case, s)
    return _exact_pages(case, s)
