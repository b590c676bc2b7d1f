"""Plain fp64 reference of the 8-bit key/value cache's operators.

Written from the definitions in include/w4a16.h, sequence by sequence and head
by head.  A cache is a dict of arrays: kc, vc uint8 [pages, H, P, D]; ks, vs
float32 [pages, H]; ranges uint8 [pages, H, 2, D]; weight float32 [pages, H, P].
Functions that write return a changed copy.
"""

from __future__ import annotations

import math

import numpy as np


def least_step(m: float) -> float:
    """The least power of two s >= 2^-100 with m <= 127 s."""
    s = 2.0 ** -100
    if m > 127 * s:
        s = 2.0 ** (math.frexp(m)[1] - 8)
        while 127 * s < m:
            s *= 2
    return s


def rescale(codes, ratio):
    return (np.rint((codes.astype(np.float64) - 128) * ratio) + 128).astype(np.uint8)


def sequences(lens, offsets):
    """(row0, n, len) of each sequence."""
    for b, length in enumerate(lens):
        if offsets is None:
            yield b, b, 1, int(length)
        else:
            yield b, int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(length)


def append_ref(cache, table, lens, offsets, k, v):
    """k, v float64 [rows, H, D]."""
    c = {n: a.copy() for n, a in cache.items()}
    H, P = c["kc"].shape[1:3]
    for b, row0, n, length in sequences(lens, offsets):
        first = length - n
        for lp in range(max(0, first) // P, (length + P - 1) // P):
            lo, hi = max(first, 0, lp * P), min(length, lp * P + P)
            if lo >= hi:
                continue
            page, a, z = table[b, lp], lo - lp * P, hi - lp * P
            for h in range(H):
                for codes, steps, x in ((c["kc"], c["ks"], k), (c["vc"], c["vs"], v)):
                    new = x[row0 + lo - first:row0 + hi - first, h]
                    step = least_step(float(np.abs(new).max()))
                    if a > 0:
                        old = float(steps[page, h])
                        step = max(step, old)
                        codes[page, h, :a] = rescale(codes[page, h, :a], old / step)
                    codes[page, h, a:z] = (np.rint(new / step) + 128).astype(np.uint8)
                    steps[page, h] = step
                c["ranges"][page, h, 0] = c["kc"][page, h, :z].min(0)
                c["ranges"][page, h, 1] = c["kc"][page, h, :z].max(0)
                c["weight"][page, h, a:z] = 0
    return c


def values(codes, steps, table_row, length, h):
    """The first `length` tokens of one sequence and head, fp64 [length, D]."""
    P = codes.shape[2]
    pages = table_row[:(length + P - 1) // P]
    x = (codes[pages, h].astype(np.float64) - 128) * steps[pages, h].astype(np.float64)[:, None, None]
    return x.reshape(-1, codes.shape[3])[:length]


def visible(pos, length, window, pages=None, P=1):
    t = np.arange(length)
    ok = t <= pos
    if window:
        ok &= t > pos - window
    if pages is not None:
        ok &= np.isin(t // P, pages)
    return ok


def attn_ref(cache, table, lens, offsets, q, scale, window=0, sel=None, n_sel=None):
    """(out, lse, spread, reach): spread = sum of p |value| per output, reach = scale times the
    largest sum of |q key| among the row's keys (what rounding errors are measured by)."""
    rows, Hq, D = q.shape
    H, P = cache["kc"].shape[1:3]
    G = Hq // H
    out, spread = np.zeros((rows, Hq, D)), np.zeros((rows, Hq, D))
    lse, reach = np.full((rows, Hq), -np.inf), np.zeros((rows, Hq))
    for b, row0, n, length in sequences(lens, offsets):
        for h in range(H):
            k = values(cache["kc"], cache["ks"], table[b], length, h)
            v = values(cache["vc"], cache["vs"], table[b], length, h)
            pages = None if sel is None else sel[b, h, :n_sel[b, h]]
            for r in range(n):
                see = visible(length - n + r, length, window, pages, P)
                if not see.any():
                    continue
                for g in range(h * G, h * G + G):
                    x = q[row0 + r, g]
                    s = scale * (k[see] @ x)
                    m = s.max()
                    p = np.exp(s - m)
                    lse[row0 + r, g] = m + math.log(p.sum())
                    p /= p.sum()
                    out[row0 + r, g] = p @ v[see]
                    spread[row0 + r, g] = p @ np.abs(v[see])
                    reach[row0 + r, g] = abs(scale) * (np.abs(k[see]) @ np.abs(x)).max()
    return out, lse, spread, reach


def weigh_ref(cache, table, lens, offsets, q, lse, scale, window=0, sel=None, n_sel=None):
    """(weight, reach): the accumulated weights fp64, and the bound's sum over what was added of
    weight times scale sum |q key|."""
    rows, Hq, D = q.shape
    H, P = cache["kc"].shape[1:3]
    G = Hq // H
    w, reach = cache["weight"].astype(np.float64), np.zeros(cache["weight"].shape)
    for b, row0, n, length in sequences(lens, offsets):
        for h in range(H):
            k = values(cache["kc"], cache["ks"], table[b], length, h)
            t = np.arange(length)
            page, slot = table[b, t // P] if length else t, t % P
            pages = None if sel is None else sel[b, h, :n_sel[b, h]]
            for r in range(n):
                see = visible(length - n + r, length, window, pages, P)
                for g in range(h * G, h * G + G):
                    l = lse[row0 + r, g]
                    if not see.any() or l == -np.inf:
                        continue
                    x = q[row0 + r, g]
                    p = np.where(see, np.exp(np.where(see, scale * (k @ x) - l, 0)), 0)
                    w[page, h, slot] += p
                    reach[page, h, slot] += p * (abs(scale) * (np.abs(k) @ np.abs(x)) + abs(l) + 1)
    return w, reach


def top(keys, count):
    """Indexes of the `count` largest keys, ties from the lowest index on, ascending."""
    order = sorted(range(len(keys)), key=lambda i: (-keys[i], i))
    return sorted(order[:count])


def select_ref(cache, table, lens, q, max_sel, sink, recent):
    rows, Hq, D = q.shape
    H, P = cache["kc"].shape[1:3]
    G = Hq // H
    sel, n_sel = np.full((rows, H, max_sel), -1, np.int32), np.zeros((rows, H), np.int32)
    for b, length in enumerate(lens):
        pages = (int(length) + P - 1) // P
        for h in range(H):
            x = q[b, h * G:h * G + G]
            up, down = np.maximum(x, 0).sum(0), np.minimum(x, 0).sum(0)
            u = least_step(float(max(up.max(), -down.min())))
            up, down = np.rint(up / u), np.rint(down / u)
            keys = []
            for i in range(pages):
                lo, hi = cache["ranges"][table[b, i], h].astype(np.float64) - 128
                keys.append(math.inf if i < sink or i >= pages - recent else
                            float(hi @ up + lo @ down) * float(cache["ks"][table[b, i], h]))
            got = top(keys, min(pages, max_sel))
            sel[b, h, :len(got)], n_sel[b, h] = got, len(got)
    return sel, n_sel


def evict_ref(cache, table, lens, dst, budget, sink, recent):
    c = {n: a.copy() for n, a in cache.items()}
    B, (H, P) = len(lens), c["kc"].shape[1:3]
    kept, new_lens = np.full((B, H, budget), -1, np.int32), np.zeros(B, np.int32)
    for b, length in enumerate(int(x) for x in lens):
        new_lens[b] = min(length, budget)
        for h in range(H):
            t = np.arange(length)
            page, slot = (table[b, t // P], t % P) if length else (t, t)
            w = cache["weight"][page, h, slot].astype(np.float64)
            keys = [math.inf if i < sink or i >= length - recent else float(w[i])
                    for i in range(length)]
            keep = np.array(top(keys, min(length, budget)), np.int64)
            kept[b, h, :len(keep)] = keep
            for j in range((len(keep) + P - 1) // P):
                part, to = keep[j * P:j * P + P], dst[b, j]
                for codes, steps, src, s0 in ((c["kc"], c["ks"], cache["kc"], cache["ks"]),
                                              (c["vc"], c["vs"], cache["vc"], cache["vs"])):
                    old = s0[page[part], h].astype(np.float64)
                    step = old.max()
                    codes[to, h, :len(part)] = rescale(src[page[part], h, slot[part]],
                                                       (old / step)[:, None])
                    steps[to, h] = step
                c["ranges"][to, h, 0] = c["kc"][to, h, :len(part)].min(0)
                c["ranges"][to, h, 1] = c["kc"][to, h, :len(part)].max(0)
                c["weight"][to, h, :len(part)] = w[part]
    return c, kept, new_lens
