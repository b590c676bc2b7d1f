"""One attention layer of a decoder on the library alone: 4-bit projections, an 8-bit cache.

    python examples/kv8_decode.py

A prompt goes through in one chunk (merged q/k/v product, append, attention over the
whole prefix, output product); then tokens one by one, each reading only the pages of
the highest score bound, its attention weights added up, and the cache cut to `budget`
tokens when it is full.  Every step's calls run in stream order without the host
looking at anything but its own counter of the length.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_only_gemv_gb300 import lib  # noqa: E402


class Layer:
    def __init__(self, hidden=2048, q_heads=8, kv_heads=2, head_dim=256, page_tokens=16,
                 max_len=4096, budget=2048, keep_pages=32, sink=4, recent=32, seed=0):
        dev, gen = "cuda", torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.hq, self.hkv, self.d = hidden, q_heads, kv_heads, head_dim
        self.scale, self.max_len, self.budget = head_dim ** -0.5, max_len, budget
        self.sink, self.recent = sink, recent
        self.gen = gen

        def weights(n, k):
            return lib.quantize(torch.randn((n, k), generator=gen, device=dev) * k ** -0.5)

        self.qkv = weights((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.o = weights(hidden, q_heads * head_dim)
        # two sets of pages: the cache and where its kept tokens go
        pages, kept = -(-max_len // page_tokens), -(-budget // page_tokens)
        n, shape = pages + kept, (kv_heads, page_tokens, head_dim)
        self.cache = lib.KV8Cache(
            *(torch.zeros((n, *shape), dtype=torch.uint8, device=dev) for _ in range(2)),
            *(torch.zeros((n, kv_heads), dtype=torch.float32, device=dev) for _ in range(2)),
            ranges=torch.zeros((n, kv_heads, 2, head_dim), dtype=torch.uint8, device=dev),
            weight=torch.zeros((n, kv_heads, page_tokens), dtype=torch.float32, device=dev))
        self.free = list(range(n))
        self.table = torch.zeros((1, pages), dtype=torch.int32, device=dev)
        self.lens = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.length, self.used, self.evictions = 0, [], 0
        self.one = lib.KV8Batch(self.table, self.lens, max_len=max_len)

        def scratch(nbytes):
            return torch.zeros(max(16, nbytes), dtype=torch.uint8, device=dev)

        self.ws_attn = scratch(lib.kv8_attn_workspace_bytes(self.cache, self.one, q_heads,
                                                            max_sel=keep_pages))
        self.ws_select = scratch(lib.kv8_select_workspace_bytes(self.cache, self.one))
        self.ws_evict = scratch(lib.kv8_evict_workspace_bytes(self.cache, self.one, budget))
        self.keep_pages, self.scratch = keep_pages, scratch
        self.ws_gemv = {m: scratch(max(lib.workspace_bytes(m, *self._nk(w)) for w in (self.qkv, self.o)))
                        for m in (1,)}

    @staticmethod
    def _nk(w):
        return w[0].shape[0], w[0].shape[1] * 8

    def tokens(self, n):
        return torch.randn((n, self.hidden), generator=self.gen, device="cuda").to(torch.bfloat16)

    def _product(self, w, x):
        m = x.shape[0]
        if m not in self.ws_gemv:
            self.ws_gemv[m] = self.scratch(max(lib.workspace_bytes(m, *self._nk(v))
                                               for v in (self.qkv, self.o)))
        return lib.gemv(*w, x, workspace=self.ws_gemv[m], status=self.status)

    def _grow(self, n):
        """Pages for n more tokens, and the length that counts them."""
        self.length += n
        p = self.cache.page_tokens
        while len(self.used) * p < self.length:
            self.used.append(self.free.pop())
            self.table[0, len(self.used) - 1] = self.used[-1]
        self.lens.fill_(self.length)

    def _split(self, x):
        rows = self._product(self.qkv, x).view(x.shape[0], self.hq + 2 * self.hkv, self.d)
        return rows[:, :self.hq], rows[:, self.hq:self.hq + self.hkv], rows[:, self.hq + self.hkv:]

    def prompt(self, x):
        """The layer's output for a prompt chunk of up to 256 tokens."""
        q, k, v = self._split(x)
        n = x.shape[0]
        self._grow(n)
        batch = lib.KV8Batch(self.table, self.lens,
                             torch.tensor([0, n], dtype=torch.int32, device="cuda"), rows=n,
                             max_new=n, max_len=self.max_len)
        lib.kv8_append(self.cache, batch, k, v, self.status)
        lse = torch.empty((n, self.hq), dtype=torch.float32, device="cuda")
        ws = self.scratch(lib.kv8_attn_workspace_bytes(self.cache, batch, self.hq))
        out = lib.kv8_attn(self.cache, batch, q, self.scale, lse=lse, workspace=ws,
                           status=self.status)
        lib.kv8_weigh(self.cache, batch, q, lse, self.scale, status=self.status)
        return self._product(self.o, out.view(n, -1))

    def step(self, x):
        """The layer's output for the next token."""
        if self.length == self.max_len or (self.length + 1) > len(self.used) * \
                self.cache.page_tokens and len(self.free) <= self._kept_pages():
            self._evict()
        q, k, v = self._split(x)
        self._grow(1)
        lib.kv8_append(self.cache, self.one, k, v, self.status)
        sel, n_sel = lib.kv8_select(self.cache, self.one, q, self.keep_pages, sink=1, recent=2,
                                    workspace=self.ws_select, status=self.status)
        lse = torch.empty((1, self.hq), dtype=torch.float32, device="cuda")
        out = lib.kv8_attn(self.cache, self.one, q, self.scale, lse=lse, sel=sel, n_sel=n_sel,
                           workspace=self.ws_attn, status=self.status)
        # the tokens of pages that were not chosen received nothing
        lib.kv8_weigh(self.cache, self.one, q, lse, self.scale, status=self.status, sel=sel,
                      n_sel=n_sel)
        self.last = dict(q=q, sel=sel, n_sel=n_sel, out=out, lse=lse)
        return self._product(self.o, out.view(1, -1))

    def _kept_pages(self):
        return -(-self.budget // self.cache.page_tokens)

    def _evict(self):
        n = self._kept_pages()
        to = [self.free.pop() for _ in range(n)]
        dst = torch.tensor([to], dtype=torch.int32, device="cuda")
        _, new_lens = lib.kv8_evict(self.cache, self.one, self.budget, dst, sink=self.sink,
                                    recent=self.recent, workspace=self.ws_evict, status=self.status)
        self.lens.copy_(new_lens)
        self.table.zero_()
        self.table[0, :n] = dst[0]
        self.free += self.used
        self.used, self.length = to, min(self.length, self.budget)
        self.evictions += 1

    def arrays(self):
        """The cache and the last step on the host (for checks)."""
        t = self.cache.tensors
        last = self.last
        names = ("kc", "vc", "ks", "vs", "ranges", "weight")
        return dict(cache={n: x.cpu().numpy() for n, x in zip(names, t)},
                    table=self.table.cpu().numpy(), lens=self.lens.cpu().numpy(),
                    q=last["q"].double().cpu().numpy(), sel=last["sel"].cpu().numpy(),
                    n_sel=last["n_sel"].cpu().numpy(), out=last["out"].double().cpu().numpy(),
                    lse=last["lse"].double().cpu().numpy())


def main():
    layer = Layer()
    x = layer.tokens(256 + 4096)
    layer.prompt(x[:256])
    for i in range(4096):
        layer.step(x[256 + i:257 + i])
    torch.cuda.synchronize()
    print(f"{layer.length} tokens cached after {layer.evictions} evictions, "
          f"status {int(layer.status.item())}")


if __name__ == "__main__":
    main()
