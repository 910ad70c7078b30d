"""Seeded states of the pool tests: page table, lengths, counts of holders and cache contents,
kept on the CPU (as the oracle changes them) and on the GPU (as the library does)."""
import numpy as np
import torch

from oracle import pool_oracle as P


class PoolPair:
    """An empty pool of `pages` pages and B rows; every call is made on both sides."""

    def __init__(self, B, max_pages, pages, *, Hkv=2, page=16, d=64, kind="bf16", seed=0, window=0):
        self.rng = np.random.default_rng(seed)
        self.B, self.M, self.pages, self.page, self.kind = B, max_pages, pages, page, kind
        self.window = window
        # entries behind a row's length may be anything
        self.table = self.rng.integers(-5, pages + 5, (B, max_pages)).tolist()
        self.lens, self.refs = [0] * B, [0] * pages
        shape = (pages, Hkv, page, d)
        if kind == "bf16":                                   # any bits: copies are bit for bit
            k, v = (self.rng.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16) for _ in "kv")
            exp = None
        else:
            k, v = (self.rng.integers(0, 256, shape).astype(np.uint8) for _ in "kv")
            exp = self.rng.integers(0, 256, shape[:3] + (2,)).astype(np.uint8)
        self.cache = [k, v, exp]
        self.to_gpu()

    def to_gpu(self):
        i32 = lambda x, *s: torch.tensor(x, dtype=torch.int32).reshape(*s).cuda()  # noqa: E731
        self.g_table = i32(self.table, self.B, self.M)
        self.g_lens, self.g_refs = i32(self.lens, self.B), i32(self.refs, self.pages)
        view = torch.bfloat16 if self.kind == "bf16" else torch.uint8
        self.g_cache = [None if x is None else torch.from_numpy(x.copy()).cuda() for x in self.cache]
        for i in (0, 1):
            self.g_cache[i] = self.g_cache[i].view(view)

    @property
    def state(self):
        return self.g_table, self.g_lens, self.g_refs

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def fork(self, ea, parents, **kw):
        self.table, self.lens, self.refs = P.fork(self.table, self.lens, self.refs, parents, self.page)
        ea.cache_fork(*self.state, self.ints(parents), page_size=self.page, **kw)

    def resize(self, ea, new_lens, window=None, **kw):
        window = self.window if window is None else window
        self.table, self.lens, self.refs, missing, copies = P.resize(
            self.table, self.lens, self.refs, new_lens, self.page, window)
        P.copy_pages(self.cache, self.cache, copies)
        got = ea.cache_resize(*self.g_cache[:2], *self.state, self.ints(new_lens),
                              kv_exp=self.g_cache[2], window=window, **kw)
        assert got.tolist() == [missing]
        return missing, copies

    def compact(self, ea, **kw):
        self.table, self.refs, used, page_map, moves = P.compact(self.table, self.lens, self.refs,
                                                                self.page)
        P.copy_pages(self.cache, self.cache, moves)
        got = ea.cache_compact(*self.g_cache[:2], *self.state, kv_exp=self.g_cache[2], **kw)
        assert got[0].tolist() == [used]
        assert got[1].tolist() == page_map
        return used, moves

    def check(self, what=""):
        torch.cuda.synchronize()
        assert self.g_lens.tolist() == self.lens, what
        assert self.g_refs.tolist() == self.refs, what
        assert np.array_equal(self.g_table.cpu().numpy().reshape(self.B, self.M),
                              np.array(self.table).reshape(self.B, self.M)), what
        for got, ref in zip(self.g_cache, self.cache):
            if ref is not None:
                view = torch.int16 if self.kind == "bf16" and got.dtype != torch.uint8 else torch.uint8
                assert np.array_equal(got.view(view).cpu().numpy(), ref), what

    def holders(self, extra=0):
        """Counts agree with the table (holders outside of it apart)."""
        n = [0] * self.pages
        for row, L in zip(self.table, self.lens):
            for e in row[:P.pages_of(L, self.page)]:
                if e >= 0:
                    n[e] += 1
        assert sum(self.refs) == sum(n) + extra and all(r >= c for r, c in zip(self.refs, n))

    def random_lens(self, most=None):
        """New lengths: some rows grow, some roll back, some end, some start."""
        cap = self.M * self.page if most is None else most
        out = []
        for row, L in zip(self.table, self.lens):
            r = self.rng.random()
            if r < 0.15:
                out.append(0)
            elif r < 0.3:
                out.append(int(self.rng.integers(0, cap + 1)))
            elif r < 0.4:
                out.append(L)
            else:
                out.append(int(np.clip(L + self.rng.integers(-9, 2 * self.page), 0, cap)))
            # a roll-back into a page that the window has given back has nothing to go on from
            if out[-1] < L and out[-1] % self.page and row[out[-1] // self.page] < 0:
                out[-1] = L
        return out

    def random_parents(self):
        return [b if r < 0.4 else -1 if r < 0.5 else int(self.rng.integers(0, self.B))
                for b, r in enumerate(self.rng.random(self.B))]
