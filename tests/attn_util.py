"""Paged caches for the attention tests: random pages on the host, their values
in fp64 by the oracle, and the same bytes on the GPU."""
import numpy as np
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from oracle import attn_ref as A


class Paged:
    """A cache of random codes; every byte that no position of a sequence holds is a NaN code (or scale)."""

    def __init__(self, fmt, hk, d, page, kv_lens, seed, *, spare=2, max_pages=None, k_gs=0.011, v_gs=0.017, pad_table=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.hk, self.d, self.page, self.rng = fmt, hk, d, page, rng
        need = [max(0, -(-n // page)) for n in kv_lens]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.max_pages = max(1, max(need, default=0)) if max_pages is None else max_pages
        self.table = np.full((len(kv_lens), self.max_pages + pad_table), 10 ** 9, dtype=np.int32)
        self.table[:, :self.max_pages] = -1
        at = 0
        for i, n in enumerate(need):
            n = min(n, self.max_pages)
            self.table[i, :n] = order[at:at + n]
            at += n
        self.gs = {"k": np.float32(k_gs if fmt == "fp8" else 0.21), "v": np.float32(v_gs if fmt == "fp8" else 0.37)}
        w = d if fmt == "fp8" else d // 2
        # row-major on the host: [page, head, position, bytes]
        shape = (self.n_pages, hk, page, w)
        self.codes, self.scales = {}, {}
        for n in "kv":
            if fmt == "fp8":
                c = A.e4m3_codes(rng.standard_normal(shape) * 60, 1.0)
                s = np.zeros((self.n_pages, hk, page, 0), np.uint8)
            else:
                c = rng.integers(0, 256, shape, dtype=np.uint8)
                s = rng.integers(0x28, 0x40, (self.n_pages, hk, page, d // 16), dtype=np.uint8)
            self.codes[n], self.scales[n] = c, s
        used = np.zeros((self.n_pages, page), bool)
        for i, n in enumerate(kv_lens):
            for p in range(min(max(n, 0), self.max_pages * page)):
                used[self.table[i, p // page], p % page] = True
        for n in "kv":
            free = np.broadcast_to(~used[:, None, :, None], self.codes[n].shape)
            if fmt == "fp8":
                self.codes[n][free] = 0x7F
            else:
                self.scales[n][np.broadcast_to(~used[:, None, :, None], self.scales[n].shape)] = 0xFF

    def place(self, i, p):
        return self.table[i, p // self.page], p % self.page

    def set_nan(self, name, i, p, head, dim):
        """Position p's value of a dim (its block, in NVFP4) becomes NaN."""
        pg, row = self.place(i, p)
        if self.fmt == "fp8":
            self.codes[name][pg, head, row, dim] = 0xFF
        else:
            self.scales[name][pg, head, row, dim // 16] = 0x7F

    def values(self, name, i, n):
        """[n, hk, d]: positions 0 .. n - 1 of sequence i."""
        p = np.arange(n)
        pg = self.table[i, p // self.page]
        return A.kv_values(self.fmt, self.codes[name][pg, :, p % self.page], self.scales[name][pg, :, p % self.page],
                           self.gs[name])

    def to(self, dev):
        """(KvCache, page table) on the GPU."""
        def t(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

        turned = {n: np.swapaxes(x[n], 2, 3) for n, x in (("v", self.codes),)}
        more = {}
        if self.fmt == "nvfp4":
            more = dict(k_scales=t(self.scales["k"]), v_scales=t(np.swapaxes(self.scales["v"], 2, 3)))
        cache = nv.KvCache(t(self.codes["k"]), t(turned["v"]), t(np.array([self.gs["k"]])), t(np.array([self.gs["v"]])),
                           format=self.fmt, **more)
        return cache, t(self.table)[:, :self.max_pages]


def i32(values, dev):
    return torch.tensor(list(values), dtype=torch.int32, device=dev)


def rows_from_cache(paged, cache):
    """The host copies of a GPU cache's arrays, row-major: (codes, scales) by name."""
    codes, scales = {}, {}
    for n in "kv":
        c = getattr(cache, n).cpu().numpy()
        codes[n] = c if n == "k" else np.swapaxes(c, 2, 3)
        if paged.fmt == "nvfp4":
            s = getattr(cache, n + "_scales").cpu().numpy()
            scales[n] = s if n == "k" else np.swapaxes(s, 2, 3)
    return codes, scales
