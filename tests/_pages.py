"""Random pools of pages for the tests of the page calls."""

import numpy as np
import torch

from bit_weight_only_gemv_gb300 import lib
from oracle import serve

ARRAYS = ("kc", "vc", "ks", "vs", "ranges", "weight")


class Pages:
    """Rows of the given lengths on scattered pages; share: row -> (row it shares whole pages with,
    how many); layers caches of one shape."""

    def __init__(self, seed, lens, P=16, H=2, D=64, layers=1, share=(), spare=6, max_pages=None,
                 pins=0, optional=True):
        rng = self.rng = np.random.default_rng(seed)
        need = [-(-n // P) for n in lens]
        mp = max_pages or max(1, max(need)) + 1
        total = max(1, sum(need) + spare)      # a pool has a page
        order = list(rng.permutation(total).astype(np.int32))
        table = np.full((len(lens), mp), -7, np.int32)
        share = dict(share)
        for b, k in enumerate(need):
            at = 0
            if b in share:
                other, at = share[b]
                table[b, :at] = table[other, :at]
            for i in range(at, k):
                table[b, i] = order.pop()
        refs = np.zeros(total, np.int32)
        for b, k in enumerate(need):
            for p in table[b, :k]:
                refs[p] += 1
        for p in order[:pins]:
            refs[p] += 1                      # kept by something else
        self.pool = serve.Pool(table, np.array(lens, np.int32), refs, P)
        self.num, self.P = total, P
        self.caches = []
        for _ in range(layers):
            c = {"kc": rng.integers(0, 256, (total, H, P, D)).astype(np.uint8),
                 "vc": rng.integers(0, 256, (total, H, P, D)).astype(np.uint8),
                 "ks": rng.random((total, H)).astype(np.float32),
                 "vs": rng.random((total, H)).astype(np.float32)}
            if optional:
                c["ranges"] = rng.integers(0, 256, (total, H, 2, D)).astype(np.uint8)
                c["weight"] = rng.random((total, H, P)).astype(np.float32)
            self.caches.append(c)

    def to_gpu(self, layered=False, most_rows=None):
        self.dev = []
        for c in self.caches:
            if layered:      # keys and values in one tensor, pages apart
                both = torch.from_numpy(np.stack([c["kc"], c["vc"]], 1)).cuda()
                kc, vc = both[:, 0], both[:, 1]
            else:
                kc, vc = (torch.from_numpy(c[k].copy()).cuda() for k in ("kc", "vc"))
            rest = {k: torch.from_numpy(c[k].copy()).cuda() for k in ARRAYS[2:] if k in c}
            self.dev.append(lib.KV8Cache(kc, vc, **rest))
        self.table, self.lens, self.refs = (
            torch.from_numpy(x.copy()).cuda() for x in (self.pool.table, self.pool.lens, self.pool.refs))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        need = lib.kv8_pages_workspace_bytes(most_rows or len(self.pool.lens), self.num)
        # the head is left as it is, and nothing is asked of the rest
        self.ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws[:4096] = 0
        return self

    def check_caches(self, copies):
        """The caches on the GPU are the host's after these copies; the next call starts from them."""
        for i, d in enumerate(self.dev):
            want = self.caches[i] = serve.copy_pages(self.caches[i], copies)
            for name, t in zip(ARRAYS, d.tensors):
                if t is not None:
                    assert np.array_equal(t.cpu().numpy(), want[name]), name
        assert not self.ws[:4096].any()

    def fork(self, parents, junk=-9):
        """Runs the call, and holds everything it gives against the reference."""
        par = np.array(parents, np.int32)
        nt = torch.full((len(par), self.table.shape[1]), junk, dtype=torch.int32, device="cuda")
        nl = torch.full((len(par),), junk, dtype=torch.int32, device="cuda")
        nr = torch.full_like(self.refs, junk)
        lib.bind_kv8_fork(self.dev, self.table, self.lens, self.refs, torch.from_numpy(par).cuda(),
                          nt, nl, nr, self.ws, self.status)()
        torch.cuda.synchronize()
        table, lens, refs, copies, errors = serve.fork(
            self.pool, parents, np.full((len(par), self.table.shape[1]), junk, np.int32))
        self.check_status(errors)
        assert np.array_equal(nl.cpu().numpy(), lens)
        if copies is None:
            self.check_caches([])
        else:
            assert np.array_equal(nt.cpu().numpy(), table)
            assert np.array_equal(nr.cpu().numpy(), refs)
            self.check_caches(copies)
        for t, old in ((self.table, self.pool.table), (self.lens, self.pool.lens),
                       (self.refs, self.pool.refs)):
            assert np.array_equal(t.cpu().numpy(), old)
        return nt, nl, nr, copies

    def reserve(self, grow=None):
        g = None if grow is None else torch.tensor(grow, dtype=torch.int32, device="cuda")
        lib.kv8_reserve(self.table, self.lens, self.refs, self.P, g, self.ws, self.status)
        torch.cuda.synchronize()
        table, lens, refs, errors = serve.reserve(self.pool, grow)
        self.check_status(errors)
        for t, want in ((self.table, table), (self.lens, lens), (self.refs, refs)):
            assert np.array_equal(t.cpu().numpy(), want)
        self.pool.table, self.pool.lens, self.pool.refs = table, lens, refs
        assert not self.ws[:4096].any()

    def compact(self, junk=-9):
        nt, nr = torch.full_like(self.table, junk), torch.full_like(self.refs, junk)
        used = torch.full((1,), junk, dtype=torch.int32, device="cuda")
        lib.bind_kv8_compact(self.dev, self.table, self.lens, self.refs, nt, nr, used, self.ws,
                             self.status)()
        torch.cuda.synchronize()
        table, refs, most, copies, errors = serve.compact(
            self.pool, np.full(self.pool.table.shape, junk, np.int32))
        self.check_status(errors)
        assert np.array_equal(nt.cpu().numpy(), table)
        assert np.array_equal(nr.cpu().numpy(), refs)
        assert int(used) == most
        self.check_caches(copies)
        for t, old in ((self.table, self.pool.table), (self.refs, self.pool.refs)):
            assert np.array_equal(t.cpu().numpy(), old)
        return nt, nr, copies

    def check_status(self, errors):
        got = int(self.status)
        assert got in {lib.STATUS_CODE["W4_ERR_" + e.upper()] for e in errors} if errors else got == 0
