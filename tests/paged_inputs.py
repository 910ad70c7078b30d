"""Seeded small inputs of the paged-cache tests: a pool, a page table and packed rows."""
import numpy as np
import torch

from oracle import paged_oracle as P


class Batch:
    """new[b] new tokens and lens[b] cached tokens per sequence, on the CPU. Slots that no
    sequence owns hold NaN (bf16) or the NaN code under exponent byte 255 (e4m3)."""

    def __init__(self, new, lens, *, Hq=4, Hkv=2, d=64, page=16, kind="bf16", seed=0,
                 spare_rows=0, k_scale=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.lens = list(new), list(lens)
        self.B, self.Hq, self.Hkv, self.d, self.page, self.kind = len(new), Hq, Hkv, d, page, kind
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + 2
        perm = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((self.B, max(1, max(need, default=0))), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.offsets[-1])
        self.T = self.rows + spare_rows
        g = torch.Generator("cpu").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q = r(self.T, Hq, d).to(torch.bfloat16)
        self.k = (r(self.T, Hkv, d) * k_scale).to(torch.bfloat16)
        self.v = (r(self.T, Hkv, d) * torch.exp2(torch.round(2 * r(self.T, Hkv, 1)))).to(torch.bfloat16)
        shape = (self.pages, Hkv, page, d)
        kc = (r(*shape) * k_scale).to(torch.bfloat16)
        vc = (r(*shape) * torch.exp2(torch.round(2 * r(*shape[:3], 1)))).to(torch.bfloat16)
        owned = np.zeros((self.pages, page), dtype=bool)
        for b, n in enumerate(lens):
            t = np.arange(n)
            owned[self.table[b, t // page], t % page] = True
        free = torch.from_numpy(~owned)
        if kind == "bf16":
            kc[free[:, None, :].expand(-1, Hkv, -1)] = float("nan")
            vc[free[:, None, :].expand(-1, Hkv, -1)] = float("nan")
            self.k_cache, self.v_cache, self.kv_exp = kc, vc, None
        else:
            (kq, ke), (vq, ve) = P.encode(kc.double().numpy()), P.encode(vc.double().numpy())
            ex = np.stack([ke, ve], axis=-1)
            mask = (~owned)[:, None, :] & np.ones((1, Hkv, 1), dtype=bool)
            kq[mask], vq[mask], ex[mask] = 127, 127, 255
            self.k_cache, self.v_cache = torch.from_numpy(kq), torch.from_numpy(vq)
            self.kv_exp = torch.from_numpy(ex)

    def cuda(self):
        t = torch.from_numpy
        d = {n: getattr(self, n).cuda() for n in ("q", "k", "v", "k_cache", "v_cache")}
        d["kv_exp"] = None if self.kv_exp is None else self.kv_exp.cuda()
        d["table"], d["offsets"] = t(self.table).cuda(), t(self.offsets).cuda()
        d["seq_lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return d

    def written(self):
        """The cache after a write of k and v: (k_cache, v_cache, kv_exp) as numpy."""
        kc, vc = self.k_cache.clone(), self.v_cache.clone()
        ex = None if self.kv_exp is None else self.kv_exp.clone()
        for b, n in enumerate(self.new):
            L, o = self.lens[b], int(self.offsets[b])
            pages, slots = P.cache_rows(self.table[b], self.page, L - n, L)
            for i, (c, x) in enumerate(((kc, self.k), (vc, self.v))):
                if ex is None:
                    c[pages, :, slots] = x[o:o + n]
                else:
                    codes, e = P.encode(x[o:o + n].double().numpy())
                    c[pages, :, slots] = torch.from_numpy(codes)
                    ex[pages, :, slots, i] = torch.from_numpy(e)
        return kc, vc, ex
