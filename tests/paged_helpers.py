"""Shared by the paged-cache tests: ragged batches over shuffled pages, the
definitions in 64 bits, and the error bounds of the kernels' arithmetic."""
import math

import numpy as np
import torch

from split_flash_decoding_kvcachescatter_gb300 import binding as B

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def least_step(dtype):
    """Largest error of one rounding below the type's normal range, where its numbers are
    evenly spaced (float16: below 2^-14, 2^-24 apart, so 2^-25)."""
    info = torch.finfo(dtype)
    return info.smallest_normal * info.eps / 2


def within(got, ref, bound, where=""):
    """Every element of got within bound of ref (64 bits), with the worst one told."""
    over = (got.double() - ref).abs() - bound
    if not bool((over <= 0).all()):  # (NaN fails too)
        at = int(torch.nan_to_num(over, nan=float("inf")).argmax())
        raise AssertionError(
            f"{where}: {int((~(over <= 0)).sum())} of {over.numel()} outside; at {at}: "
            f"{float(got.flatten()[at])!r} for {float(ref.flatten()[at])!r}, bound "
            f"{float(bound.expand_as(ref).reshape(-1)[at]):.3g}")


class Paged:
    """A batch of sequences (n new tokens from position p each) over pages in
    shuffled order.  Pages' rows that hold no live key are NaN, and so are the
    pages that no sequence uses; the table's unused entries (columns of them behind
    the longest sequence) are out of range."""

    def __init__(self, n, p, H, Hkv, D, dtype, page, seed=0, spare=3, tail_rows=0,
                 columns=2):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.n, self.p, self.H, self.Hkv, self.D, self.page = n, p, H, Hkv, D, page
        self.dtype = DTYPES[dtype]
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
        self.k_pages = torch.full(shape, math.nan, dtype=self.dtype, device=DEV)
        self.v_pages = torch.full(shape, math.nan, dtype=self.dtype, device=DEV)
        self.k, self.v = [], []
        for i in range(M):
            L = n[i] + p[i] if n[i] else 0
            k, v = (torch.empty(Hkv, L, D, device=DEV).normal_(generator=g).to(self.dtype)
                    for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            for j in range(need[i]):
                a, b = j * page, min(L, (j + 1) * page)
                self.k_pages[self.table_host[i, j], :, :b - a] = k[:, a:b]
                self.v_pages[self.table_host[i, j], :, :b - a] = v[:, a:b]
        self.q = torch.empty(self.rows, H, D, device=DEV).normal_(generator=g).to(self.dtype)
        self.offsets_host = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.positions = torch.tensor(p, dtype=torch.int32, device=DEV)
        self.row_offsets = torch.from_numpy(self.offsets_host).to(DEV)
        self.page_table = torch.from_numpy(self.table_host).to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.cache = B.PagedCache(self.k_pages, self.v_pages)
        self.batch = B.PagedBatch(self.positions, self.row_offsets, self.page_table, self.rows,
                                  max([1] + n))
        self.workspace = B.paged_attention_workspace(self.cache, self.batch, H)

    def attend(self, out=None, q=None, **kw):
        out = torch.full((self.rows, self.H, self.D), 7.0, dtype=self.dtype, device=DEV) \
            if out is None else out
        B.kvs_paged_attention(self.q if q is None else q, self.cache, self.batch, out,
                              workspace=self.workspace, d_status=self.status, **kw)
        return out

    def reference(self):
        """(out, bound) in 64 bits: bound is what the kernel's arithmetic may be off by."""
        G = self.H // self.Hkv
        u = half_step(self.dtype)
        f32 = self.dtype == torch.float32
        out = torch.full((self.rows, self.H, self.D), 7.0, dtype=torch.float64, device=DEV)
        bound = torch.zeros_like(out)
        for i, (n, p) in enumerate(zip(self.n, self.p)):
            if n == 0:
                continue
            a = int(self.offsets_host[i])
            q = self.q[a:a + n].double().view(n, self.Hkv, G, self.D)
            k, v = self.k[i].double(), self.v[i].double()
            L = n + p
            s = torch.einsum("tged,gld->gtel", q, k) / math.sqrt(self.D)
            size = torch.einsum("tgd,gld->gtl", q.abs().amax(2), k.abs()).amax() / math.sqrt(self.D)
            far = torch.arange(L, device=DEV)[None] > (p + torch.arange(n, device=DEV))[:, None]
            w = torch.softmax(s.masked_fill(far[None, :, None], -math.inf), -1)
            o = torch.einsum("gtel,gld->tged", w, v).reshape(n, self.H, self.D)
            vmax = v.abs().amax()
            # scores: products exact in 16 bits, 3 x 2^-21 (two truncated low parts and the
            # dropped low x low) in float32; sums of D products, each addition 2^-23 (the
            # tensor cores may truncate), D / 8 sequential groups of three products; the
            # exponent's rounding and ex2 add 2^-22 of the exponent and 2^-22
            ds = size * ((3 * 2.0 ** -21 if f32 else 0) + 3 * self.D / 8 * 2.0 ** -23 + 2.0 ** -22)
            rel = 2 * ds + 2.0 ** -22
            # weights times v: one rounding of each weight to the type (float32: split, 3 x
            # 2^-21); weights under 2^-14 of float16 are off by 2^-25 at most, and the row's
            # largest is 1; the sum over L / 8 steps (three products each in float32), and
            # that of the weights
            rel += (3 * 2.0 ** -21 if f32 else u) + (L * 2.0 ** -25 if self.dtype == torch.float16 else 0)
            rel += ((3 * L / 8 if f32 else L / 16) + L / 8 + 64) * 2.0 ** -23
            out[a:a + n] = o
            bound[a:a + n] = rel * vmax + u * (o.abs() + rel * vmax) + least_step(self.dtype)
        return out, bound

    def check(self, got, where=""):
        ref, bound = self.reference()
        assert int(self.status.item()) == 0, where
        within(got, ref, bound, where)


def row_of(offsets, r):
    return int(np.searchsorted(offsets[1:], r, side="right"))
