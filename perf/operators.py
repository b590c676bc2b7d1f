"""The 8-bit key/value cache's operators: plain forms, the library's calls, and the cases that time them.

A decoder layer's attention runs between the 4-bit projections: the merged
q/k/v product writes the new tokens' rows, the cache stores keys and values in
8 bits with one step for each (page of tokens, head), and attention reads
them.  Five operators:

append   new rows into the pages, each touched block's step grown (and its
         older codes rescaled) when a new value needs it
attn     attention of the new tokens over their sequence, single tokens and
         prompt chunks, causal, optionally within a sliding window
sparse   the pages with the highest score bound for a token, and attention
         over those alone
weigh    the attention weight that each cached token received, added up
evict    the tokens of most accumulated weight (and the first and last ones)
         gathered into fresh pages

The format: value = (code - 128) * step, code uint8 [pages][heads][tokens of
a page][head size], step fp32 [pages][heads], a power of two when the cache's
own writer chose it.  Steps that are powers of two make every code a whole
number that does not depend on the width of the arithmetic, so codes are
returned as they are stored, beside their steps, and have to be equal.
"""

import math

import torch

own = False

_DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of eight running conversations
        dict(name="append-token", op="append", B=8, n=1, L=4096, Hkv=8, D=128, P=32),
        # sixteen prompts of different lengths, a chunk of up to 256 tokens each
        dict(name="append-chunks", op="append", B=16, n=256, L=2048, Hkv=8, D=128, P=64),
        # batch-1 decode on a sliding layer: 8 query heads on 2 key heads of 256 (the
        # hidden-2048 decode pass: q 2048 rows, k and v 512 rows), 512-token window
        dict(name="attn-token", op="attn", B=1, n=1, L=700, Hq=8, Hkv=2, D=256, P=16, window=512),
        # a serving batch of 24 conversations of different lengths
        dict(name="attn-batch", op="attn", B=24, n=1, L=16384, Hq=64, Hkv=8, D=128, P=32, window=0),
        # the last 256-token chunk of a 16k prompt
        dict(name="attn-chunk", op="attn", B=1, n=256, L=16384, Hq=32, Hkv=8, D=128, P=64, window=0),
        # six prompts' chunks on a sliding layer, small heads, three query heads a key head
        dict(name="attn-chunks-window", op="attn", B=6, n=200, L=6000, Hq=24, Hkv=8, D=64, P=16,
             window=1024),
        # one long conversation, 48 pages of 32 tokens read out of 1024
        dict(name="sparse-token", op="sparse", B=1, n=1, L=32768, Hq=16, Hkv=4, D=128, P=32,
             max_sel=48),
        # sixteen long conversations
        dict(name="sparse-batch", op="sparse", B=16, n=1, L=32768, Hq=32, Hkv=8, D=128, P=32,
             max_sel=128),
        # one decoded token's weights in a batch of eight
        dict(name="weigh-token", op="weigh", B=8, n=1, L=16384, Hq=32, Hkv=8, D=128, P=32,
             window=0),
        # a prompt chunk's weights, two prompts
        dict(name="weigh-chunk", op="weigh", B=2, n=256, L=8192, Hq=32, Hkv=8, D=128, P=64,
             window=0),
        # one short conversation cut to 1000 tokens
        dict(name="evict-one", op="evict", B=1, L=3000, Hkv=2, D=256, P=16, budget=1000),
        # a batch cut from up to 16k tokens to 4096 each
        dict(name="evict-batch", op="evict", B=8, L=16384, Hkv=8, D=128, P=32, budget=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "sparse", "weigh", "evict"])
    D, P, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8, 8, 16])
    chunk = rng.random() < 0.5
    c = dict(op=op, Hkv=Hkv, D=D, P=P)
    if op == "append":
        c.update(B=_log(rng, 1, 16), n=_log(rng, 2, 256) if chunk else 1)
        c["L"] = c["n"] + _log(rng, 1, 4000)
        return c
    if op == "evict":
        c.update(B=_log(rng, 1, 8), L=_log(rng, 200, 16000))
        c["budget"] = max(96, _log(rng, 96, 4096))
        return c
    c["Hq"] = Hkv * G
    if op == "sparse":
        c.update(B=_log(rng, 1, 16), n=1, L=_log(rng, 1000, 32768), max_sel=_log(rng, 4, 128))
        while c["B"] * Hkv * c["L"] * D > 2 ** 29:
            c["B"] = max(1, c["B"] // 2)
            c["L"] = max(1000, c["L"] * 3 // 4)
        return c
    if chunk:
        c.update(B=_log(rng, 1, 6), n=_log(rng, 2, 256))
        c["L"] = c["n"] + _log(rng, 1, 16000)
        c["window"] = rng.choice([0, 0, 128, 777, 1024])
        most = 2 ** 34 if op == "attn" else 2 ** 33          # rows x keys x head size
        while c["B"] * c["n"] * c["L"] * c["Hq"] * D > most:
            c["B"] = max(1, c["B"] // 2)
            c["L"] = c["n"] + max(1, (c["L"] - c["n"]) * 2 // 3)
            c["n"] = max(2, c["n"] * 3 // 4)
    else:
        c.update(B=_log(rng, 1, 32), n=1, L=_log(rng, 1, 32768))
        c["window"] = rng.choice([0, 0, 0, 512, 1000])
        while c["B"] * Hkv * c["L"] * D > 2 ** 28:
            c["B"] = max(1, c["B"] // 2)
            c["L"] = max(1, c["L"] * 3 // 4)
    return c


def _news(c):
    """New tokens of each sequence: the first has n, the others fewer."""
    n = c.get("n", 1)
    return [n if b == 0 or n == 1 else 1 + (n * (37 * b % 61)) // 61 for b in range(c["B"])]


def _lens(c):
    """Tokens of each sequence, the new ones among them: the first has L, the others L/4 to L."""
    L = c["L"]
    return [L if b == 0 else max(m, L - (3 * L * (29 * b % 53)) // (4 * 53))
            for b, m in enumerate(_news(c))]


def _seen(c):
    """(query, key) pairs of each sequence, and the keys that any of its queries sees."""
    w = c.get("window", 0) or (1 << 60)
    pairs = [sum(min(w, p + 1) for p in range(L - n, L)) for n, L in zip(_news(c), _lens(c))]
    keys = [min(L, n - 1 + w) for n, L in zip(_news(c), _lens(c))]
    return pairs, keys


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    c, op = case, case["op"]
    D, P, H, B = c["D"], c["P"], c["Hkv"], c["B"]
    T = sum(_news(c))
    if op == "append":
        # bf16 rows in, codes out, a step and a range row of each touched block, its weights
        blocks = sum((L - 1) // P - (L - n) // P + 1 for n, L in zip(_news(c), _lens(c))) * H
        return {"bytes": T * H * D * 2 * (2 + 1) + blocks * (2 * 4 + 2 * D) + T * H * 4, "flops": 0}
    if op == "attn":
        pairs, keys = _seen(c)
        q = T * c["Hq"] * D
        return {"bytes": 2 * sum(keys) * H * D + 2 * sum(keys) // P * H * 4 + 4 * q + T * c["Hq"] * 4,
                "flops": 4 * sum(pairs) * c["Hq"] * D}
    if op == "sparse":
        pages = [-(-L // P) for L in _lens(c)]
        kept = sum(min(L, P * c["max_sel"]) for L in _lens(c))
        return {"bytes": sum(pages) * H * (2 * D + 4) + 2 * kept * H * D
                + B * c["Hq"] * (6 * D + 4) + B * H * c["max_sel"] * 4,
                "flops": 4 * sum(pages) * H * D + 4 * kept * c["Hq"] * D}
    if op == "weigh":
        pairs, keys = _seen(c)
        return {"bytes": sum(keys) * H * (D + 8) + T * c["Hq"] * (2 * D + 4),
                "flops": 2 * sum(pairs) * c["Hq"] * D}
    kept = sum(min(L, c["budget"]) for L in _lens(c)) * H
    return {"bytes": sum(_lens(c)) * H * 4 + 2 * kept * (2 * D + 4) + kept * 4, "flops": 0}


# ------------------------------------------------------------------ inputs
def _pow2_step(m):
    """The smallest power of two s with m <= 127 s, at least 2^-100 (m fp32, >= 0)."""
    f, e = torch.frexp(m)
    e = torch.where(f <= 127 / 128, e - 7, e - 6)
    e = torch.where(m > 0, e, -100).clamp(min=-100).to(torch.int32)
    return ((e + 127) << 23).view(torch.float32)      # its bits: exact on every device


def _filled(gen, pages, H, P, D, spread):
    """Codes and steps of random keys or values: normal, channels of unequal size."""
    codes = torch.empty((pages, H, P, D), dtype=torch.uint8, device=_DEV)
    steps = torch.empty((pages, H), dtype=torch.float32, device=_DEV)
    size = torch.exp(spread * torch.randn((H, 1, D), generator=gen, device=_DEV))
    each = max(1, 2 ** 26 // (H * P * D))
    for i in range(0, pages, each):
        x = torch.randn((min(each, pages - i), H, P, D), generator=gen, device=_DEV) * size
        s = _pow2_step(x.abs().amax((2, 3)))
        steps[i:i + each] = s
        codes[i:i + each] = (torch.round(x / s[:, :, None, None]) + 128).to(torch.uint8)
    return codes, steps


def prepare(case, seed):
    c = case
    op, B, H, D, P = c["op"], c["B"], c["Hkv"], c["D"], c["P"]
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    news, lens = _news(c), _lens(c)
    mp = max(-(-L // P) for L in lens)
    used = sum(-(-L // P) for L in lens)
    extra = B * (-(-c["budget"] // P)) if op == "evict" else 0
    num = used + extra + 3
    order = torch.randperm(num, generator=gen, device=_DEV).to(torch.int32)
    table = torch.full((B, mp), -1, dtype=torch.int32, device=_DEV)
    at = 0
    for b, L in enumerate(lens):
        k = -(-L // P)
        table[b, :k] = order[at:at + k]
        at += k
    offs = [0]
    for n in news:
        offs.append(offs[-1] + n)
    s = dict(case=c, table=table, T=offs[-1], max_new=max(news), max_len=max(lens),
             lens=torch.tensor(lens, dtype=torch.int32, device=_DEV),
             offs=torch.tensor(offs, dtype=torch.int32, device=_DEV))
    s["kc"], s["ks"] = _filled(gen, num, H, P, D, 0.4)
    s["vc"], s["vs"] = _filled(gen, num, H, P, D, 0.2)
    if op in ("append", "sparse", "evict"):
        # lowest and highest key code of each channel over a page's tokens
        pos = torch.arange(mp * P, device=_DEV).view(1, mp, P)
        live = torch.zeros((num, P), dtype=torch.bool, device=_DEV)
        before = s["lens"] - (s["offs"][1:] - s["offs"][:-1] if op == "append" else 0)
        sel = table >= 0
        live[table[sel].long()] = (pos < before[:, None, None])[sel]
        lo, hi = s["kc"].new_full((1,), 255), s["kc"].new_zeros(1)
        m = live[:, None, :, None]
        s["ranges"] = torch.stack([torch.where(m, s["kc"], lo).amin(2),
                                   torch.where(m, s["kc"], hi).amax(2)], 2).contiguous()
    if op in ("append", "weigh", "evict"):
        # accumulated weights: most tokens little, some much, many none at all
        w = torch.exp(2 * torch.randn((num, H, P), generator=gen, device=_DEV) - 4)
        s["weight"] = w * (torch.rand((num, H, P), generator=gen, device=_DEV) < 0.9)
    if op == "append":
        # rows of a merged q/k/v product with as many query heads again: strided views
        qkv = torch.randn((s["T"], 3 * H, D), generator=gen, device=_DEV)
        qkv = (qkv * torch.exp(0.5 * torch.randn((s["T"], 3 * H, 1), generator=gen, device=_DEV)))
        s["qkv"] = qkv.to(torch.bfloat16)
        s["k"], s["v"] = s["qkv"][:, H:2 * H], s["qkv"][:, 2 * H:]
    if op in ("attn", "sparse", "weigh"):
        Hq = c["Hq"]
        q = torch.randn((s["T"], Hq, D), generator=gen, device=_DEV)
        q = q * torch.exp(0.3 * torch.randn((1, Hq, 1), generator=gen, device=_DEV))
        s["q"], s["scale"] = q.to(torch.bfloat16), D ** -0.5
        s["out"] = torch.empty((s["T"], Hq, D), dtype=torch.bfloat16, device=_DEV)
        s["lse"] = torch.empty((s["T"], Hq), dtype=torch.float32, device=_DEV)
        if op == "weigh":
            s["lse"] = _plain_attn(s)["lse"]
    if op == "sparse":
        s["sel"] = torch.empty((B, H, c["max_sel"]), dtype=torch.int32, device=_DEV)
        s["n_sel"] = torch.empty((B, H), dtype=torch.int32, device=_DEV)
    if op == "evict":
        npd = -(-c["budget"] // P)
        s["dst"] = order[used:used + B * npd].view(B, npd).contiguous()
        s["kept"] = torch.empty((B, H, c["budget"]), dtype=torch.int32, device=_DEV)
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device=_DEV)
    return s


# forced pages of a sparse call, forced tokens of an eviction
_SINK_PAGES, _RECENT_PAGES = 1, 2
_SINK, _RECENT = 4, 64


# ------------------------------------------------------------------ plain forms
def _rows(s):
    """Index of each sequence's new rows in the packed ones [B, max_new], which of them exist,
    and their positions."""
    n = s["offs"][1:] - s["offs"][:-1]
    i = torch.arange(s["max_new"], device=_DEV)[None]
    real = i < n[:, None]
    at = (s["offs"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    return at, real, (s["lens"] - n)[:, None] + i


def _softmax_over(scores, mask, v):
    """Output, and log of the sum of exponentials, of masked rows (none left: 0 and -inf)."""
    scores = torch.where(mask, scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    out = torch.where(l > 0, (p @ v) / l, 0.0)
    return out, (m + torch.log(l)).squeeze(-1)


def _scores(s):
    """Scaled scores [B, H, n * G, keys] and which of them count."""
    c = s["case"]
    B, H, D, P, G = c["B"], c["Hkv"], c["D"], c["P"], c["Hq"] // c["Hkv"]
    pages = s["table"].clamp(min=0).long()
    keys = (s["kc"][pages].float() - 128) * s["ks"][pages][..., None, None]
    keys = keys.transpose(1, 2).reshape(B, H, -1, D)
    at, real, pos = _rows(s)
    q = s["q"].float()[at].view(B, s["max_new"], H, G, D).transpose(1, 2).reshape(B, H, -1, D)
    kpos = torch.arange(keys.shape[2], device=_DEV)
    sees = (kpos <= pos[..., None]) & real[..., None]
    if c.get("window", 0):
        sees &= kpos > pos[..., None] - c["window"]
    mask = sees[:, None, :, None, :].expand(B, 1, s["max_new"], G, -1).reshape(B, 1, -1, kpos.numel())
    return (q @ keys.transpose(2, 3)) * s["scale"], mask, pages


def _packed(s, x):
    """[B, H, n * G, ...] back to the packed rows [T, Hq, ...]."""
    c = s["case"]
    B, H, G = c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    x = x.view(B, H, s["max_new"], G, *x.shape[3:]).transpose(1, 2).flatten(0, 1).flatten(1, 2)
    n = s["offs"][1:] - s["offs"][:-1]
    row = torch.arange(s["T"], device=_DEV, dtype=torch.int32)
    b = torch.searchsorted(s["offs"][1:].contiguous(), row, right=True)
    return x[b * s["max_new"] + (row - s["offs"][b])].contiguous()


def _plain_attn(s):
    c = s["case"]
    scores, mask, pages = _scores(s)
    v = (s["vc"][pages].float() - 128) * s["vs"][pages][..., None, None]
    v = v.transpose(1, 2).reshape(c["B"], c["Hkv"], -1, c["D"])
    out, lse = _softmax_over(scores, mask, v)
    return {"out": _packed(s, out).to(torch.bfloat16), "lse": _packed(s, lse)}


def _plain_append(s):
    c = s["case"]
    B, H, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    n = s["offs"][1:] - s["offs"][:-1]
    start, end = s["lens"] - n, s["lens"]
    nt = (s["max_new"] + P - 2) // P + 1
    lp = (start // P)[:, None] + torch.arange(nt, device=_DEV)
    lp = torch.minimum(lp, ((end - 1).clamp(min=0) // P)[:, None])
    page = s["table"].gather(1, lp.long()).clamp(min=0).long()                   # [B, nt]
    pos = lp[..., None] * P + torch.arange(P, device=_DEV)                       # [B, nt, P]
    new = (pos >= start[:, None, None]) & (pos < end[:, None, None])
    old = pos < start[:, None, None]
    row = (s["offs"][:-1, None, None] + pos - start[:, None, None]).clamp(0, s["T"] - 1).long()
    newm, oldm = new[:, :, None, :, None], old[:, :, None, :, None]
    some = new.any(-1)[..., None]

    def put(codes, steps, x):
        was, s0 = codes[page], steps[page]                                       # [B, nt, H, P, D]
        vals = x.float()[row].transpose(2, 3)
        m = torch.where(newm, vals.abs(), 0.0).amax((3, 4))
        step = torch.maximum(torch.where(old.any(-1)[..., None], s0, 0.0), _pow2_step(m))
        again = torch.round((was.float() - 128) * (s0 / step)[..., None, None]) + 128
        fresh = torch.round(vals / step[..., None, None]) + 128
        got = torch.where(newm, fresh, torch.where(oldm, again, was.float()))
        got = torch.where(some[..., None, None], got, was.float()).to(torch.uint8)
        codes[page] = got
        steps[page] = torch.where(some, step, s0)
        return got

    k = put(s["kc"], s["ks"], s["k"])
    put(s["vc"], s["vs"], s["v"])
    live = newm | oldm
    rng = torch.stack([torch.where(live, k, k.new_full((1,), 255)).amin(3),
                       torch.where(live, k, k.new_zeros(1)).amax(3)], 3)
    s["ranges"][page] = torch.where(some[..., None, None], rng, s["ranges"][page])
    s["weight"][page] = torch.where(new[:, :, None, :], 0.0, s["weight"][page])
    return {k: s[k] for k in ("kc", "ks", "vc", "vs", "ranges", "weight")}


def _top(key, count, valid):
    """Indexes of the `count` largest along the last axis, ties to the lowest index, ascending,
    -1 past the valid ones (valid [..., 1]: how many entries count)."""
    at = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :count]
    n = valid.clamp(max=count)
    i = torch.arange(at.shape[-1], device=_DEV)
    at = torch.sort(torch.where(i < n, at, 1 << 40), dim=-1).values
    at = torch.where(at < 1 << 40, at, -1).to(torch.int32)
    return torch.nn.functional.pad(at, (0, count - at.shape[-1]), value=-1), n


def _plain_sparse(s):
    c = s["case"]
    B, H, D, P, G, S = c["B"], c["Hkv"], c["D"], c["P"], c["Hq"] // c["Hkv"], c["max_sel"]
    q = s["q"].float().view(B, H, G, D)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)                      # [B, H, D]
    step = _pow2_step(torch.maximum(up, -down).amax(-1, keepdim=True))
    up, down = torch.round(up / step), torch.round(down / step)
    pages = s["table"].clamp(min=0).long()
    r = s["ranges"][pages].float() - 128                                         # [B, mp, H, 2, D]
    score = (r[:, :, :, 1] * up[:, None]).sum(-1) + (r[:, :, :, 0] * down[:, None]).sum(-1)
    score = (score * s["ks"][pages]).transpose(1, 2)                             # [B, H, mp]
    np_ = ((s["lens"] + P - 1) // P)[:, None, None]
    i = torch.arange(score.shape[-1], device=_DEV)
    forced = (i < _SINK_PAGES) | (i >= np_ - _RECENT_PAGES)
    key = torch.where(i < np_, torch.where(forced, math.inf, score), -math.inf)
    sel, n_sel = _top(key, S, np_.expand(B, H, 1))
    pg = torch.gather(pages, 1, sel.clamp(min=0).long().view(B, -1)).view(B, H, S)
    h = torch.arange(H, device=_DEV)[None, :, None]
    keys = ((s["kc"][pg, h].float() - 128) * s["ks"][pg, h][..., None, None]).flatten(2, 3)
    vals = ((s["vc"][pg, h].float() - 128) * s["vs"][pg, h][..., None, None]).flatten(2, 3)
    pos = (sel[..., None] * P + torch.arange(P, device=_DEV)).flatten(2)         # [B, H, S * P]
    sees = (sel >= 0).repeat_interleave(P, -1) & (pos < s["lens"][:, None, None])
    out, lse = _softmax_over((q @ keys.transpose(2, 3)) * s["scale"], sees[:, :, None], vals)
    return {"out": out.reshape(B, H * G, D).to(torch.bfloat16), "lse": lse.reshape(B, H * G),
            "sel": sel, "n_sel": n_sel[..., 0].to(torch.int32)}


def _plain_weigh(s):
    c = s["case"]
    B, H, P, G = c["B"], c["Hkv"], c["P"], c["Hq"] // c["Hkv"]
    scores, mask, pages = _scores(s)
    at, real, _ = _rows(s)
    lse = s["lse"][at].view(B, s["max_new"], H, G).transpose(1, 2).reshape(B, H, -1, 1)
    p = torch.where(mask, torch.exp(scores - lse), 0.0).sum(2)                   # [B, H, keys]
    p = p.view(B, H, -1, P).transpose(1, 2)
    s["weight"].index_put_((pages,), p, accumulate=True)
    return {"weight": s["weight"]}


def _plain_evict(s):
    c = s["case"]
    B, H, D, P, K = c["B"], c["Hkv"], c["D"], c["P"], c["budget"]
    pages = s["table"].clamp(min=0).long()
    w = s["weight"][pages].transpose(1, 2).reshape(B, H, -1)
    pos, n = torch.arange(w.shape[-1], device=_DEV), s["lens"][:, None, None]
    forced = (pos < _SINK) | (pos >= n - _RECENT)
    kept, cnt = _top(torch.where(pos < n, torch.where(forced, math.inf, w), -math.inf), K,
                     n.expand(B, H, 1))
    npd = s["dst"].shape[1]
    at = torch.nn.functional.pad(kept, (0, npd * P - K), value=-1)               # [B, H, npd * P]
    live = (at >= 0).view(B, H, npd, P)
    src = torch.gather(pages, 1, (at.clamp(min=0) // P).long().view(B, -1)).view(B, H, -1)
    slot, h = (at.clamp(min=0) % P).long(), torch.arange(H, device=_DEV)[None, :, None]
    dst = s["dst"].long()
    any_ = live.any(-1).transpose(1, 2)                                          # [B, npd, H]
    lv = live.transpose(1, 2)                                                    # [B, npd, H, P]

    def move(codes, steps):
        u = codes[src, h, slot].view(B, H, npd, P, D).transpose(1, 2).float() - 128
        s0 = steps[src, h].view(B, H, npd, P).transpose(1, 2)
        step = torch.where(lv, s0, 0.0).amax(-1, keepdim=True)
        got = (torch.round(u * (s0 / step)[..., None]) + 128).nan_to_num(128.0).to(torch.uint8)
        got = torch.where(lv[..., None], got, codes[dst])
        codes[dst] = got
        steps[dst] = torch.where(any_, step[..., 0], steps[dst])
        return got

    k = move(s["kc"], s["ks"])
    move(s["vc"], s["vs"])
    m = lv[..., None]
    rng = torch.stack([torch.where(m, k, k.new_full((1,), 255)).amin(3),
                       torch.where(m, k, k.new_zeros(1)).amax(3)], 3)
    s["ranges"][dst] = torch.where(any_[..., None, None], rng, s["ranges"][dst])
    wm = s["weight"][src, h, slot].view(B, H, npd, P).transpose(1, 2)
    s["weight"][dst] = torch.where(lv, wm, s["weight"][dst])
    s["kept"], s["new_lens"] = kept, cnt[:, 0, 0].to(torch.int32)
    return {k: s[k] for k in ("kc", "ks", "vc", "vs", "ranges", "weight", "kept", "new_lens")}


_PLAIN = {"append": _plain_append, "attn": _plain_attn, "sparse": _plain_sparse,
          "weigh": _plain_weigh, "evict": _plain_evict}


# ------------------------------------------------------------------ the library's calls
def _bound(s):
    """The calls of a serving loop on these buffers, marshalled once, as such a loop keeps them."""
    from bit_weight_only_gemv_gb300 import lib

    c, op = s["case"], s["case"]["op"]
    cache = lib.KV8Cache(s["kc"], s["vc"], s["ks"], s["vs"], ranges=s.get("ranges"),
                         weight=s.get("weight"))
    batch = lib.KV8Batch(s["table"], s["lens"], None if s["max_new"] == 1 else s["offs"],
                         max_new=s["max_new"], max_len=s["max_len"])

    def scratch(nbytes):
        return torch.zeros(max(16, nbytes), dtype=torch.uint8, device=_DEV)

    if op == "append":
        return [lib.bind_kv8_append(cache, batch, s["k"], s["v"])]
    if op == "attn":
        ws = scratch(lib.kv8_attn_workspace_bytes(cache, batch, c["Hq"]))
        return [lib.bind_kv8_attn(cache, batch, s["q"], s["scale"], s["out"], lse=s["lse"],
                                  window=c["window"], workspace=ws)]
    if op == "sparse":
        ws = scratch(lib.kv8_select_workspace_bytes(cache, batch))
        wa = scratch(lib.kv8_attn_workspace_bytes(cache, batch, c["Hq"], max_sel=c["max_sel"]))
        return [lib.bind_kv8_select(cache, batch, s["q"], s["sel"], s["n_sel"], sink=_SINK_PAGES,
                                    recent=_RECENT_PAGES, workspace=ws),
                lib.bind_kv8_attn(cache, batch, s["q"], s["scale"], s["out"], lse=s["lse"],
                                  sel=s["sel"], n_sel=s["n_sel"], workspace=wa)]
    if op == "weigh":
        return [lib.bind_kv8_weigh(cache, batch, s["q"], s["lse"], s["scale"],
                                   window=c["window"])]
    ws = scratch(lib.kv8_evict_workspace_bytes(cache, batch, c["budget"]))
    return [lib.bind_kv8_evict(cache, batch, s["dst"], s["kept"], s["new_lens"], sink=_SINK,
                               recent=_RECENT, workspace=ws)]


_GIVES = {"append": ("kc", "ks", "vc", "vs", "ranges", "weight"), "attn": ("out", "lse"),
          "sparse": ("out", "lse", "sel", "n_sel"), "weigh": ("weight",),
          "evict": ("kc", "ks", "vc", "vs", "ranges", "weight", "kept", "new_lens")}


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
def _sequence(s, b, h):
    """Keys and values of one sequence and head, fp64 [tokens, D]."""
    P, L = s["case"]["P"], int(s["lens"][b])
    pg = s["table"][b, :-(-L // P)].long()
    k = (s["kc"][pg, h].double() - 128) * s["ks"][pg, h].double()[:, None, None]
    v = (s["vc"][pg, h].double() - 128) * s["vs"][pg, h].double()[:, None, None]
    return k.flatten(0, 1)[:L], v.flatten(0, 1)[:L], pg


def _each(s):
    """(sequence, head, its rows' slice, their positions, query rows fp64 [n, G, D])."""
    c = s["case"]
    G, offs, lens = c["Hq"] // c["Hkv"], s["offs"].tolist(), s["lens"].tolist()
    for b in range(c["B"]):
        rows = slice(offs[b], offs[b + 1])
        pos = torch.arange(lens[b] - offs[b + 1] + offs[b], lens[b], device=_DEV)
        for h in range(c["Hkv"]):
            yield b, h, rows, pos, s["q"][rows, h * G:(h + 1) * G].double()


def _visible(s, pos, keys):
    i = torch.arange(keys, device=_DEV)
    ok = i[None] <= pos[:, None]
    w = s["case"].get("window", 0)
    return ok & (i[None] > pos[:, None] - w) if w else ok


def _least_step(m):
    """Block by block: the least power of two, from 2^-100 on, that holds m in 127 steps."""
    e = torch.floor(torch.log2((m / 127).clamp(min=2.0 ** -99))).to(torch.int64) - 1
    s = ((e + 1023) << 52).view(torch.float64)
    s = torch.where(127 * s < m, 2 * s, s)
    s = torch.where(127 * s < m, 2 * s, s)
    return torch.where(127 * s < m, 2 * s, s)


def _exact_append(s):
    """Steps and weights block by block (the codes have no value but the stored one)."""
    c, P = s["case"], s["case"]["P"]
    got = {k: s[k].double() for k in ("ks", "vs", "weight")}
    offs, lens = s["offs"].tolist(), s["lens"].tolist()
    for b in range(c["B"]):
        first = lens[b] - (offs[b + 1] - offs[b])
        for lp in range(first // P, (lens[b] - 1) // P + 1):
            lo, hi = max(first, lp * P), min(lens[b], (lp + 1) * P)
            pg, at = int(s["table"][b, lp]), offs[b] + lo - first
            got["weight"][pg, :, lo % P:(hi - 1) % P + 1] = 0
            for name, x in (("ks", s["k"]), ("vs", s["v"])):
                need = _least_step(x[at:at + hi - lo].double().abs().amax((0, 2)))
                got[name][pg] = torch.maximum(got[name][pg], need) if lo % P else need
    return {"kc": None, "vc": None, "ranges": None, **got}


def _exact_evict(s):
    c, P, K = s["case"], s["case"]["P"], s["case"]["budget"]
    got = {k: s[k].double() for k in ("ks", "vs", "weight")}
    lens = s["lens"].tolist()
    for b in range(c["B"]):
        pg, L = s["table"][b].long(), lens[b]
        for h in range(c["Hkv"]):
            w = s["weight"][pg[:-(-L // P)], h].double().flatten()[:L]
            rank = w.clone()
            rank[:_SINK] = rank[max(0, L - _RECENT):] = math.inf
            keep = torch.topk(rank, min(K, L)).indices       # one set of several where weights tie:
            low = rank[keep].min()                           # the border's lowest indexes
            sure, tied = (rank > low).nonzero()[:, 0], (rank == low).nonzero()[:, 0]
            keep = torch.cat([sure, tied[:min(K, L) - sure.numel()]]).sort().values
            for j in range(-(-keep.numel() // P)):
                part, to = keep[j * P:(j + 1) * P], int(s["dst"][b, j])
                got["weight"][to, h, :part.numel()] = w[part]
                for name in ("ks", "vs"):
                    got[name][to, h] = s[name][pg[part // P], h].double().max()
    return {"kc": None, "vc": None, "ranges": None, "kept": None, "new_lens": None, **got}


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "append":
        return _exact_append(s)
    if op == "evict":
        return _exact_evict(s)
    G = c["Hq"] // c["Hkv"]
    if op == "weigh":
        w = s["weight"].double()
        for b, h, rows, pos, q in _each(s):
            k, _, pg = _sequence(s, b, h)
            dots = torch.einsum("tgd,kd->tgk", q, k) * s["scale"]
            p = torch.exp(dots - s["lse"][rows, h * G:(h + 1) * G].double()[..., None])
            p = (p * _visible(s, pos, k.shape[0])[:, None]).sum((0, 1))
            full = torch.zeros(pg.numel() * c["P"], dtype=torch.float64, device=_DEV)
            full[:p.numel()] = p
            w[pg, h] += full.view(-1, c["P"])
        return {"weight": w}
    out = torch.zeros((s["T"], c["Hq"], c["D"]), dtype=torch.float64, device=_DEV)
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=_DEV)
    picked = _plain_sparse(s)["sel"].tolist() if op == "sparse" else None
    for b, h, rows, pos, q in _each(s):
        k, v, pg = _sequence(s, b, h)
        see = _visible(s, pos, k.shape[0])
        if picked is not None:
            member = torch.zeros(pg.numel(), dtype=torch.bool, device=_DEV)
            member[[i for i in picked[b][h] if i >= 0]] = True
            see = see & member.repeat_interleave(c["P"])[:k.shape[0]]
        dots = (torch.einsum("tgd,kd->tgk", q, k) * s["scale"]).masked_fill(~see[:, None], -math.inf)
        out[rows, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", torch.softmax(dots, -1), v)
        lse[rows, h * G:(h + 1) * G] = torch.logsumexp(dots, -1)
    r = {"out": out, "lse": lse}
    return r if op == "attn" else {**r, "sel": None, "n_sel": None}
