"""Plain fp64 references of routing, expert sums and logit rules (w4_route, w4_moe_combine,
w4_logits_adjust), and of the page calls (w4_kv8_fork, w4_kv8_reserve, w4_kv8_compact), written from
include/w4a16.h with loops where loops say it best."""

import numpy as np


# ------------------------------------------------------------------ routing
def scores(x, sigmoid):
    x = np.asarray(x, np.float64)
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    e = np.exp(x - x.max())
    return e / e.sum()


def route_row(x, bias, k, groups, top_groups, best, sigmoid, renorm, scale):
    """(ids, weights) of one token, or None where it is refused."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (bias is not None and not np.isfinite(bias).all()) or \
            (not sigmoid and np.isinf(x.max())):
        return None
    s = scores(x, sigmoid)
    c = s if bias is None else s + np.asarray(bias, np.float64)
    order = x if bias is None else c
    size = len(x) // groups
    allowed = range(groups)
    if top_groups < groups:
        def group_score(g):
            part = slice(g * size, (g + 1) * size)
            if best == 1 and bias is None:
                return x[part].max()
            top = np.sort(c[part])[::-1][:best]
            return top[0] + top[1] if len(top) == 2 else top[0]
        allowed = sorted(range(groups), key=lambda g: (-group_score(g), g))[:top_groups]
    can = [e for e in range(len(x)) if e // size in set(allowed)]
    ids = sorted(can, key=lambda e: (-order[e], e))[:k]
    w = s[ids]
    if renorm:
        if sigmoid:   # relative to the largest, in logs: small scores keep their ratios
            w = np.exp(-np.logaddexp(0.0, -x[ids]) + np.logaddexp(0.0, -x[ids].max())) \
                if x[ids].max() > -np.inf else np.zeros(k)
        else:
            w = np.exp(x[ids] - x[ids].max()) if x[ids].max() > -np.inf else np.zeros(k)
        w = w / w.sum() if w.sum() > 0 else np.zeros(k)
    return np.array(ids, np.int32), scale * w


def combine(y, weights, add):
    """(out, sum of magnitudes), fp64."""
    T, k = weights.shape
    prod = weights[..., None].astype(np.float64) * y.reshape(T, k, -1).astype(np.float64)
    out, size = prod.sum(1), np.abs(prod).sum(1)
    if add is not None:
        out, size = out + add, size + np.abs(add)
    return out, size


# ------------------------------------------------------------------ logits
def adjust_row(x, tokens=(), prompt=0, repetition=1.0, presence=0.0, frequency=0.0, bias=(),
               mask=None):
    """(logits fp64, sum of magnitudes, which were named): bias is a list of (id, value)."""
    out = np.asarray(x, np.float64).copy()
    size = np.abs(out)
    named = np.zeros(len(out), bool)
    counts = {}
    for i, v in enumerate(tokens):
        counts[v] = counts.get(v, 0) + (i >= prompt)
    last = dict(bias)                     # a token named twice: the later entry
    for v, n in counts.items():
        named[v] = True
        out[v] = out[v] / repetition if out[v] > 0 else out[v] * repetition
        size[v] = abs(out[v])
        if n:
            out[v] -= frequency * n + presence
            size[v] += abs(frequency * n) + abs(presence)
    for v, b in last.items():
        named[v] = True
        out[v] += b
        size[v] += abs(b)
    if mask is not None:
        out[~mask] = -np.inf
        named |= ~mask
    return out, size, named


# ------------------------------------------------------------------ pages
class Pool:
    """Table, lengths and references of a batch on a pool, as the calls see them."""

    def __init__(self, table, lens, refs, P):
        self.table, self.lens, self.refs, self.P = table.copy(), lens.copy(), refs.copy(), P

    def pages_of(self, b):
        """Pages that row b names, or None where it breaks its bounds."""
        n = int(self.lens[b])
        if n < 0 or n > self.table.shape[1] * self.P:
            return None
        row = [int(p) for p in self.table[b, :-(-n // self.P)]]
        return row if all(0 <= p < len(self.refs) for p in row) else None


def fork(pool, parents, new_table):
    """(new table, new lens, new refs, copies [(from, to, tokens)], errors); new_table: what the
    entries past a row's pages hold.  Copies None: too few free pages."""
    rows = [pool.pages_of(b) for b in range(len(pool.lens))]
    errors = {"index"} if any(r is None for r in rows) else set()
    table, refs = new_table.copy(), pool.refs.copy()
    lens = np.zeros(len(parents), np.int32)
    gone = [rows[b] for b in range(len(parents), len(rows)) if rows[b] is not None]
    come = []
    for b, p in enumerate(parents):
        if p < -1 or p >= len(rows) or (p >= 0 and rows[p] is None):
            lens[b] = -1
            errors.add("index")
            continue
        if b < len(rows) and rows[b] is not None:
            gone.append(rows[b])
        if p >= 0:
            come.append((b, rows[p]))
            lens[b] = pool.lens[p]
            table[b, :len(rows[p])] = rows[p]
    for r in gone:
        for p in r:
            refs[p] -= 1
    for _, r in come:
        for p in r:
            refs[p] += 1
    ends = {}
    for b, r in come:
        if lens[b] % pool.P:
            ends.setdefault(r[-1], []).append(b)
    todo = sorted(b for p, who in ends.items()
                  for b in (who[1:] if len(who) == refs[p] else who))
    free = [p for p in range(len(refs)) if refs[p] == 0]
    if len(free) < len(todo):
        return table, np.full(len(parents), -1, np.int32), refs, None, errors | {"state"}
    copies = []
    for b, to in zip(todo, free):
        at = -(-int(lens[b]) // pool.P) - 1
        copies.append((int(table[b, at]), to, int(lens[b]) % pool.P))
        table[b, at] = to
    for a, to, _ in copies:
        refs[a] -= 1
        refs[to] = 1
    return table, lens, refs, copies, errors


def reserve(pool, grow):
    """(table, lens, refs, errors) after the call."""
    errors, want = set(), []
    for b, n in enumerate(int(x) for x in pool.lens):
        g = int(n > 0) if grow is None else int(grow[b])
        most = pool.table.shape[1] * pool.P
        if g < 0 or not 0 <= n <= most or n + g > most:
            errors.add("index")
            continue
        want.append((b, -(-n // pool.P), -(-(n + g) // pool.P), n + g))
    free = [p for p in range(len(pool.refs)) if pool.refs[p] == 0]
    if len(free) < sum(e - a for _, a, e, _ in want):
        return pool.table, pool.lens, pool.refs, errors | {"state"}
    table, lens, refs = pool.table.copy(), pool.lens.copy(), pool.refs.copy()
    free = iter(free)
    for b, a, e, n in want:
        for i in range(a, e):
            table[b, i] = next(free)
            refs[table[b, i]] = 1
        lens[b] = n
    return table, lens, refs, errors


def compact(pool, new_table):
    """(new table, new refs, used, copies, errors)."""
    rows = [pool.pages_of(b) for b in range(len(pool.lens))]
    errors = {"index"} if any(r is None for r in rows) else set()
    named = np.zeros(len(pool.refs), np.int64)
    for r in rows:
        for p in r or ():
            named[p] += 1
    n = int((pool.refs != 0).sum())
    src = [p for p in range(n, len(named)) if pool.refs[p] != 0 and named[p] == pool.refs[p]]
    holes = [p for p in range(n) if pool.refs[p] == 0]
    to = {a: b for a, b in zip(src, holes)}
    refs = pool.refs.copy()
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    table = new_table.copy()
    for b, r in enumerate(rows):
        if r is not None:
            table[b, :len(r)] = [to.get(p, p) for p in r]
    used = int(np.nonzero(refs)[0].max()) + 1 if refs.any() else 0
    return table, refs, used, [(a, b, pool.P) for a, b in to.items()], errors


def copy_pages(cache, copies):
    """The cache's arrays (dict, as in w4_kv8_cache) after the copies."""
    got = {k: v.copy() for k, v in cache.items()}
    for a, b, n in copies:
        for k in ("kc", "vc", "weight"):
            if k in got:
                got[k][b, :, :n] = cache[k][a, :, :n]
        for k in ("ks", "vs", "ranges"):
            if k in got:
                got[k][b] = cache[k][a]
    return got
