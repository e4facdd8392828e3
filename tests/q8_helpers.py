"""Shared by the tests of the 8-bit paged cache: batches over pages of e4m3 numbers with a scale a
block, the definitions in 64 bits, and the error bounds of the kernels' arithmetic."""
import math

import numpy as np
import torch

from paged_helpers import DEV, DTYPES, half_step, least_step, within
from split_flash_decoding_kvcachescatter_gb300 import binding as B

E4M3 = torch.float8_e4m3fn
BLOCK = B.KVS_SCALE_BLOCK


def e4m3(x):
    """x (64 bits) to the nearest e4m3 number, ties to even, 448 at most."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def scale_of(most):
    """The least power of two (2^-60 at least) under which `most` (64 bits) is 448 at most."""
    m, e = torch.frexp(most.clamp_min(2.0 ** -200))  # m 2^e, and 448 is 0.875 2^9
    return torch.exp2((e - 9 + (m > 0.875)).clamp_min(-60).double())


def numbers(shape, g, device=DEV):
    """e4m3 numbers as a cache holds them: a block's largest near the top of the range."""
    x = torch.empty(shape, device=device).normal_(generator=g) * 110
    return x.clamp(-448, 448).to(E4M3)


class PagedQ8:
    """A batch of sequences (n new tokens from position p each) over pages in shuffled order.  Rows
    that hold no live key are NaN numbers, blocks without one have NaN scales, and so have the pages
    that no sequence uses; the table's unused entries are out of range.  `spread`: scales are 2^k,
    k even over +-spread around that of values near 1."""

    def __init__(self, n, p, H, Hkv, D, dtype, page, seed=0, spare=3, tail_rows=0, columns=2,
                 spread=1, powers=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.n, self.p, self.H, self.Hkv, self.D, self.page = n, p, H, Hkv, D, page
        self.dtype, self.powers = DTYPES[dtype], powers
        M = len(n)
        need = [-(-(a + b) // page) if a else 0 for a, b in zip(n, p)]
        total = sum(need) + spare
        order = rng.permutation(total)
        self.table_host = np.full((M, max(need + [1]) + columns), -1, np.int32)
        at = 0
        for i in range(M):
            self.table_host[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
        self.rows = sum(n) + tail_rows
        shape = (total, Hkv, page, D)
        dead = torch.full(shape, 0x7f, dtype=torch.uint8, device=DEV)
        self.k_pages, self.v_pages = dead.view(E4M3), dead.clone().view(E4M3)
        self.k_scales, self.v_scales = (torch.full((total, Hkv, page // BLOCK), math.nan, device=DEV)
                                        for _ in range(2))
        self.k, self.v = [], []
        for i in range(M):
            L = n[i] + p[i] if n[i] else 0
            for pages, scales, kept in ((self.k_pages, self.k_scales, self.k),
                                        (self.v_pages, self.v_scales, self.v)):
                x = numbers((Hkv, L, D), g)
                e = rng.integers(-spread, spread + 1, (Hkv, -(-L // BLOCK)))
                s = 2.0 ** (e - 7.0) * (1 if powers else rng.uniform(1, 2, e.shape))
                s = torch.from_numpy(s.astype(np.float32)).to(DEV)
                for j in range(need[i]):
                    a, b = j * page, min(L, (j + 1) * page)
                    at = int(self.table_host[i, j])
                    pages.view(torch.uint8)[at, :, :b - a] = x[:, a:b].view(torch.uint8)
                    c, d = a // BLOCK, -(-b // BLOCK)
                    scales[at, :, :d - c] = s[:, c:d]
                kept.append(x.double() * s.double().repeat_interleave(BLOCK, 1)[:, :L, None])
        self.q = torch.empty(self.rows, H, D, device=DEV).normal_(generator=g).to(self.dtype)
        self.offsets_host = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.positions = torch.tensor(p, dtype=torch.int32, device=DEV)
        self.row_offsets = torch.from_numpy(self.offsets_host).to(DEV)
        self.page_table = torch.from_numpy(self.table_host).to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.cache = B.PagedCacheQ8(self.k_pages, self.v_pages, self.k_scales, self.v_scales)
        self.batch = B.PagedBatch(self.positions, self.row_offsets, self.page_table, self.rows,
                                  max([1] + n))
        self.workspace = B.paged_attention_q8_workspace(self.cache, self.batch, H)

    def attend(self, out=None, q=None, **kw):
        out = torch.full((self.rows, self.H, self.D), 7.0, dtype=self.dtype, device=DEV) \
            if out is None else out
        B.kvs_paged_attention_q8(self.q if q is None else q, self.cache, self.batch, out,
                                 workspace=self.workspace, d_status=self.status, **kw)
        return out

    def reference(self):
        """(out, bound) in 64 bits: bound is what the kernel's arithmetic may be off by."""
        G = self.H // self.Hkv
        u = half_step(self.dtype)
        f32 = self.dtype == torch.float32
        two = f32 or max(self.n) * G <= 16  # weights as two float16 parts
        out = torch.full((self.rows, self.H, self.D), 7.0, dtype=torch.float64, device=DEV)
        bound = torch.zeros_like(out)
        for i, (n, p) in enumerate(zip(self.n, self.p)):
            if n == 0:
                continue
            a = int(self.offsets_host[i])
            q = self.q[a:a + n].double().view(n, self.Hkv, G, self.D)
            k, v = self.k[i], self.v[i]
            L = n + p
            s = torch.einsum("tged,gld->gtel", q, k) / math.sqrt(self.D)
            size = torch.einsum("tgd,gld->gtl", q.abs().amax(2), k.abs()).amax() / math.sqrt(self.D)
            far = torch.arange(L, device=DEV)[None] > (p + torch.arange(n, device=DEV))[:, None]
            w = torch.softmax(s.masked_fill(far[None, :, None], -math.inf), -1)
            o = torch.einsum("gtel,gld->tged", w, v).reshape(n, self.H, self.D)
            # |value| under the weights: blocks may differ much in size
            vs = v.abs().amax(2)
            vmean = torch.einsum("gtel,gl->tge", w, vs).reshape(n, self.H, 1)
            vmax = vs.amax()
            lg = torch.log2(vmax / vs.amin().clamp_min(1e-30)).abs() + 10
            # scores: q exact in 16 bits (2^-39 of the largest element a term), two parts of 22
            # bits in float32; stored numbers exact; sums of D products in steps of 16 (two in
            # float32), each addition 2^-23 (the tensor cores may truncate) and 16 of them in a
            # step; three factors of 2^-24
            ds = size * ((2.0 ** -22 if f32 else 0) + self.D * 2.0 ** -39 + 3 * self.D / 8 * 2.0 ** -23
                         + 2.0 ** -22)
            # chunks in 16 bits: numbers times their block's scale over the tile's, which for powers
            # of two rounds what is 2^-33 of the largest or less, else twice to float16 (2^-12 each)
            if not two:
                ds += size * (2.0 ** -26 if self.powers else 2.0 ** -11)
            # exponents x + (log2 scale - m): sums of numbers of at most 1.5 size + lg, each
            # rounded to 2^-24 of itself; ex2 2^-22
            ds += 2 * (1.5 * size + lg) * 2.0 ** -24
            rel = 2 * ds + 2.0 ** -21
            # weights: a rounding to float16 (2^-12), or two parts (2^-22); the sums over L / 16
            # steps and that of the weights
            rel = rel + (2.0 ** -22 if two else 2.0 ** -12 if self.powers else 3 * 2.0 ** -12) + (L / 16 * 2 + L / 8 + 64) * 2.0 ** -23
            # weights that float16 no longer holds: 2^-25 beside 2^10 (2^5 in chunks)
            lost = L * vmax * 2.0 ** (-35 if two else -30)
            out[a:a + n] = o
            err = rel * vmean + lost
            bound[a:a + n] = err + u * (o.abs() + err) + least_step(self.dtype)
        return out, bound

    def check(self, got, where=""):
        ref, bound = self.reference()
        assert int(self.status.item()) == 0, where
        within(got, ref, bound, where)
