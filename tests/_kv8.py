"""Random caches and batches for the kv8 tests, on the host and on the GPU."""

import numpy as np
import torch

from bit_weight_only_gemv_gb300 import lib


def bf16_round(x):
    """fp64 array rounded to bf16 values."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy()


class Case:
    """Sequences of the given lengths and new-row counts on scattered pages (news None: one row
    each, no offsets)."""

    def __init__(self, seed, lens, news, H, D, P, G=1, spare=3, pow2=True):
        rng = np.random.default_rng(seed)
        self.H, self.D, self.P, self.G = H, D, P, G
        self.lens = np.array(lens, np.int32)
        self.offsets = None if news is None else np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.rows = len(lens) if news is None else int(sum(news))
        self.max_new = 1 if news is None else max(1, max(news))
        need = [-(-x // P) for x in lens]
        self.max_pages = max(1, max(need))
        n = sum(need) + spare
        order = rng.permutation(n).astype(np.int32)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.free = order[at:]
        scale = np.exp(rng.normal(size=(n, H))) * 0.02
        steps = (2.0 ** np.rint(np.log2(scale))) if pow2 else scale
        c = {"kc": rng.integers(0, 256, (n, H, P, D)).astype(np.uint8),
             "vc": rng.integers(0, 256, (n, H, P, D)).astype(np.uint8),
             "ks": steps.astype(np.float32),
             "vs": (steps[::-1] * 2).astype(np.float32),
             "weight": np.abs(rng.normal(size=(n, H, P))).astype(np.float32)}
        c["ranges"] = np.stack([c["kc"].min(2), c["kc"].max(2)], 2)
        self.cache = c
        self.q = bf16_round(rng.normal(size=(self.rows, H * G, D)))
        self.scale = D ** -0.5
        self.rng = rng

    def fix_ranges(self, lens=None):
        """Ranges over the tokens that exist (as the writers keep them)."""
        for b, n in enumerate(self.lens if lens is None else lens):
            for i in range(-(-int(n) // self.P)):
                z = min(self.P, int(n) - i * self.P)
                pg = self.table[b, i]
                self.cache["ranges"][pg, :, 0] = self.cache["kc"][pg, :, :z].min(1)
                self.cache["ranges"][pg, :, 1] = self.cache["kc"][pg, :, :z].max(1)

    # ---- the GPU's side
    def to_gpu(self, max_len=None, layered=False):
        """layered: kc and vc are views of one tensor [pages, 2, H, P, D] (padded strides)."""
        c = self.cache
        if layered:
            both = torch.from_numpy(np.stack([c["kc"], c["vc"]], 1)).cuda()
            kc, vc = both[:, 0], both[:, 1]
        else:
            kc, vc = torch.from_numpy(c["kc"]).cuda(), torch.from_numpy(c["vc"]).cuda()
        rest = {n: torch.from_numpy(c[n]).cuda() for n in ("ks", "vs", "ranges", "weight")}
        self.dev = lib.KV8Cache(kc, vc, **rest)
        self.batch = lib.KV8Batch(
            torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda(),
            None if self.offsets is None else torch.from_numpy(self.offsets).cuda(),
            rows=self.rows, max_new=self.max_new,
            max_len=int(self.lens.max()) if max_len is None else max_len)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self.dev, self.batch

    def gpu_q(self):
        return torch.from_numpy(self.q.astype(np.float32)).cuda().to(torch.bfloat16)

    def dev_arrays(self):
        t = self.dev.tensors
        return {n: x.cpu().numpy() for n, x in zip(("kc", "vc", "ks", "vs", "ranges", "weight"), t)}

    def scratch(self, nbytes):
        return torch.zeros(max(16, nbytes), dtype=torch.uint8, device="cuda")

    def attn(self, window=0, sel=None, n_sel=None, q=None):
        """(out fp64, lse fp64) of one kv8_attn call, outputs poisoned before."""
        q = self.gpu_q() if q is None else q
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        ws = self.scratch(lib.kv8_attn_workspace_bytes(
            self.dev, self.batch, q.shape[1], max_sel=0 if sel is None else sel.shape[-1]))
        lib.kv8_attn(self.dev, self.batch, q, self.scale, out, lse, window, sel, n_sel, ws,
                     self.status)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()


def score_error(D, reach):
    """Bound of a score's error: exact products, fp32 sums of D of them (chunks of 16 with one
    truncation each at worst), two more fp32 roundings, against sum |q key|."""
    return (D / 8 + 8) * 2.0 ** -23 * reach


def check_attn(got_out, got_lse, ref, D):
    """|out - ref| within the bounds of: score errors d (each weight off by a factor e^+-d, so by
    2 d against the normalised sum), weights rounded to fp16 (2^-11), running rescales and
    exponentials (2^-18 in all), sums of fp32, one bf16 rounding (2^-9, a whole ulp allowed)."""
    out, lse, spread, reach = ref
    d = score_error(D, reach)
    tol = (2 * d + 2.0 ** -10)[..., None] * spread + 2.0 ** -8 * np.abs(out) + 1e-30
    bad = ~(np.abs(got_out - out) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got_out[bad][:4], out[bad][:4], tol[bad][:4])
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(got_out[empty] == 0)
    ltol = d[~empty] + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse[~empty])
    assert np.all(np.abs(got_lse[~empty] - lse[~empty]) <= ltol)
