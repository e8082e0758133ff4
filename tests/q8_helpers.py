"""Batches of the 8-bit cache's attention, run on the GPU and held against the oracle."""
import math

import numpy as np
import torch

from oracle import q8_oracle as Q
from ranking_prefill_gb300 import lib

BF16 = torch.bfloat16


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Batch:
    """A cache filled by rows of a size of their own, everything unused NaN, and
    the queries of each request's newest rows."""

    def __init__(self, lens, ns, hq, hkv, D, page=16, order="rows", seed=0, spread=0.5, scale=0.0, pad=0,
                 max_rows=None, extra_T=0, max_pages=None):
        r = np.random.default_rng(seed)
        self.lens, self.ns, self.hq, self.hkv, self.D, self.page = list(lens), list(ns), hq, hkv, D, page
        B = len(self.lens)
        pages = [-(-l // page) for l in self.lens]
        self.n_pages = sum(pages) + 3
        perm = r.permutation(self.n_pages)
        self.max_pages = max_pages or max(max(pages), 1)
        self.table = np.full((B, self.max_pages), -7, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = perm[at:at + pages[b]]
            at += pages[b]
        shape = (self.n_pages, page, hkv)
        kv = []
        for _ in range(2):
            x = r.standard_normal(shape + (D,)) * 2.0 ** (spread * r.standard_normal(shape + (1,)) * 2)
            e = Q.exponent(x)
            c = Q.codes(x, e)
            kv += [c, (e + 127).astype(np.uint8)]
        used = np.zeros(shape[:2], bool)
        for b, l in enumerate(self.lens):
            for p in range(l):
                used[self.table[b, p // page], p % page] = True
        for c, e in (kv[:2], kv[2:]):
            c[~used] = Q.NAN_CODE
            e[~used] = r.integers(0, 256, e[~used].shape)
        self.kc, self.ke, self.vc, self.ve = kv
        self.cu = np.concatenate([[0], np.cumsum(self.ns)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_T
        self.q = torch.as_tensor(r.standard_normal((self.T, hq, D))).to(BF16)
        self.scale, self.order, self.pad = scale, order, pad
        self.max_rows = max_rows or max(max(self.ns), 1)

    def cache(self):
        def codes(c):
            t = torch.as_tensor(c).cuda()
            if self.order == "heads":
                return t.transpose(1, 2).contiguous().transpose(1, 2)
            return t
        exps = lambda e: torch.as_tensor(np.ascontiguousarray(e.transpose(0, 2, 1))).cuda()  # noqa: E731
        if self.order == "both":                           # K and V rows side by side in one buffer
            kv = torch.stack([torch.as_tensor(self.kc), torch.as_tensor(self.vc)], dim=3).cuda()
            return lib.PagedCacheQ8(kv[:, :, :, 0], kv[:, :, :, 1], exps(self.ke), exps(self.ve))
        return lib.PagedCacheQ8(codes(self.kc), codes(self.vc), exps(self.ke), exps(self.ve))

    def put(self):
        """Device tensors of a call."""
        D, hq = self.D, self.hq
        self.c = self.cache()
        self.desc = lib.PagedAttentionDesc(self.c, B=len(self.lens), T=self.T, Hq=hq, max_rows=self.max_rows,
                                           scale=self.scale)
        w = hq * D + self.pad

        def rows(fill):
            return torch.full((max(self.T, 1), w), fill, dtype=BF16, device="cuda")[:, :hq * D].unflatten(1, (hq, D))
        self.dq, self.o = rows(0.0), rows(7.0)
        self.dq[:self.T] = self.q.cuda()
        self.lse = torch.full((hq, self.T), 7.0, device="cuda")
        self.dt, self.dl, self.dc = i32(self.table), i32(self.lens), i32(self.cu)
        self.ws = torch.full((self.desc.workspace_size(),), 0xA5, dtype=torch.uint8, device="cuda")
        return self

    def call(self, stream=None):
        lib.mis_paged_attention_q8_fwd(self.desc, self.dq, self.o, self.lse, self.dt, self.dl, self.dc, self.ws,
                                       stream=stream)
        return self

    def run(self):
        self.put().call()
        torch.cuda.synchronize()
        assert lib.mis_get_device_status(self.ws) == lib.MIS_OK
        return self

    def gathered(self, b):
        """Values of request b's rows [L, hkv, D]; rows of pages outside the cache as NaN."""
        at = np.arange(self.lens[b])
        page = self.table[b, at // self.page]
        ok = (page >= 0) & (page < self.n_pages)
        safe = np.where(ok, page, 0)
        k = Q.values(self.kc[safe, at % self.page], self.ke[safe, at % self.page])
        v = Q.values(self.vc[safe, at % self.page], self.ve[safe, at % self.page])
        k[~ok] = np.nan
        v[~ok] = 0.0
        return k, v

    def check(self, skip=()):
        """Every row against the oracle. A score is a sum of D products in fp32 (D
        roundings of at most the sum of their sizes, and the tensor core may cut
        instead of round: twice that), scaled by three more; the exponential is
        good to 2^-21. P is rounded to 11 bits (2^-11 of its size); held in steps
        of 2^-24 where its largest is 2^11 at least, it is off by 2^-36 of the largest
        weight for keys that weigh little. Each of l products may be cut at 2^-24 of
        the largest as fp32 adds it. o is rounded to bf16."""
        o, lse, q = f64(self.o), f64(self.lse), f64(self.q)
        scale = self.scale or 1.0 / math.sqrt(self.D)
        for b, (l, n) in enumerate(zip(self.lens, self.ns)):
            r0 = int(self.cu[b])
            if b in skip:
                assert (o[r0:r0 + n] == 7).all()
                continue
            k, v = self.gathered(b)
            ro, rl, av, big = Q.attention(q[r0:r0 + n], k, v, n, scale)
            ds = big * ((2 * self.D + 8) * 2.0 ** -24) + 2.0 ** -20      # of a score, natural logarithm
            tol = 2.0 ** -8 * np.abs(ro) + av * (2.0 ** -11 + 2 * ds[..., None]) + l * 2.0 ** -24 * np.nan_to_num(
                np.abs(v)).max(initial=0.0) + 1e-30
            got = o[r0:r0 + n]
            assert (np.isnan(got) == np.isnan(ro)).all(), (b, np.isnan(got).sum(), np.isnan(ro).sum())
            bad = ~(np.abs(got - ro) <= tol) & ~np.isnan(ro)
            assert not bad.any(), (b, l, n, np.argwhere(bad)[:5], np.abs(got - ro)[bad][:5], tol[bad][:5])
            gl = lse[:, r0:r0 + n].T
            assert (np.isneginf(gl) == np.isneginf(rl)).all() and (np.isnan(gl) == np.isnan(rl)).all()
            fine = np.isfinite(rl)
            assert (np.abs(gl[fine] - rl[fine]) <= (2 * ds + np.abs(rl) * 2.0 ** -22 + 2.0 ** -19)[fine]).all(), b
        end = int(self.cu[-1])
        assert (o[end:] == 7).all() and (lse[:, end:] == 7).all()
        return self
