"""kvs_rope_scatter_paged_q8 against the definition in 64 bits: numbers, scales, what grows and what
is left as it was; and the whole way from rows to attention."""
import math

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, half_step, least_step, within
from q8_helpers import BLOCK, E4M3, PagedQ8, e4m3, scale_of
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


class Append:
    """Sequences with n new tokens from position p each; the cache holds older numbers everywhere,
    under scales of 2^-9 to 2^-6.  Rows of q, k and v are column blocks of one matrix."""

    def __init__(self, n, p, H, Hkv, D, dtype, page, rot=None, interleaved=False, seed=0, tail_rows=0,
                 scale=1.0, size=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.n, self.p, self.H, self.Hkv, self.D, self.page = n, p, H, Hkv, D, page
        self.dtype, self.rot, self.il, self.scale = DTYPES[dtype], D if rot is None else rot, interleaved, scale
        M = len(n)
        need = [-(-(a + b) // page) for a, b in zip(n, p)]
        order, at = rng.permutation(sum(need) + 3), 0
        self.table = np.full((M, max(need) + 2), -1, np.int32)
        for i in range(M):
            self.table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
        self.rows = sum(n) + tail_rows
        shape = (len(order), Hkv, page, D)
        self.pages, self.scales = [], []
        for _ in range(2):
            x = (torch.empty(shape, device=DEV).normal_(generator=g) * 100).clamp(-448, 448).to(E4M3)
            self.pages.append(x)
            k = torch.from_numpy(rng.integers(-9, -5, (shape[0], Hkv, page // BLOCK))).to(DEV)
            self.scales.append(torch.exp2(k.float()))
        qkv = size * torch.empty(self.rows, (H + 2 * Hkv) * D, device=DEV).normal_(generator=g)
        # blocks of very different size, so that scales grow here and stay there
        qkv *= torch.exp2(torch.from_numpy(rng.integers(-4, 5, (self.rows, 1))).to(DEV).float())
        qkv = qkv.to(self.dtype)
        self.q = qkv[:, :H * D].unflatten(1, (H, D))
        self.k = qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
        self.v = qkv[:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
        self.offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        w = 10000.0 ** (-np.arange(self.rot // 2) * 2.0 / max(self.rot, 1))
        self.inv_freq = torch.from_numpy(w.astype(np.float32)).to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.positions = torch.tensor(p, dtype=torch.int32, device=DEV)
        self.row_offsets = torch.from_numpy(self.offsets).to(DEV)
        self.page_table = torch.from_numpy(self.table).to(DEV)
        self.batch = B.PagedBatch(self.positions, self.row_offsets, self.page_table, self.rows,
                                  max([1] + n))

    def cache(self):
        return B.PagedCacheQ8(self.pages[0], self.pages[1], self.scales[0], self.scales[1])

    def run(self, q_out=None, **kw):
        out = torch.full((self.rows, self.H, self.D), 7.0, dtype=self.dtype, device=DEV) \
            if q_out is None else q_out
        B.kvs_rope_scatter_paged_q8(self.q, self.k, self.v, out, self.cache(), self.batch,
                                    self.inv_freq, interleaved=self.il, scale=self.scale,
                                    d_status=self.status, **kw)
        return out

    def turned(self, x):
        pos = np.concatenate([np.arange(a, a + b) for a, b in zip(self.p, self.n)] or [[]])
        x = x[:len(pos)].double().clone()
        t = torch.from_numpy(pos).to(DEV).double()[:, None] * self.inv_freq.double()
        c, s = self.scale * t.cos()[:, None], self.scale * t.sin()[:, None]
        half = self.rot // 2
        a = slice(0, self.rot, 2) if self.il else slice(0, half)
        b = slice(1, self.rot, 2) if self.il else slice(half, self.rot)
        u, v = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = u * c - v * s, v * c + u * s
        return x

    def check(self):
        before = [t.clone() for t in self.pages], [t.clone() for t in self.scales]
        out = self.run()
        assert int(self.status.item()) == 0
        total = int(self.offsets[-1])
        ref = self.turned(self.q)
        # cos, sin, two products and their sum in float32 (2^-24 each, of |a| + |b|), the angle to
        # 2^-31 of pi; then one rounding
        u = half_step(self.dtype)
        big = self.q[:total].double().abs().amax(-1, keepdim=True) * 2 * self.scale
        err = 4 * 2.0 ** -23 * big
        within(out[:total], ref, err + u * (ref.abs() + err) + least_step(self.dtype), "q")
        assert (out[total:] == 7).all()
        for kind, x in ((0, self.turned(self.k)), (1, self.v[:total].double())):
            numbers, scales = before[0][kind], before[1][kind]
            got, gscale = self.pages[kind], self.scales[kind]
            slack = (4 * 2.0 ** -23 * 2 * self.scale * self.k[:total].double().abs().amax(-1, keepdim=True)
                     if kind == 0 else 0 * x[..., :1])
            want_n, want_s = numbers.double().clone(), scales.double().clone()
            tol = torch.zeros_like(want_n)
            for i, (n, p) in enumerate(zip(self.n, self.p)):
                a = p
                while a < p + n:
                    b = min(p + n, a // BLOCK * BLOCK + BLOCK)
                    at, lo = int(self.table[i, a // self.page]), a % self.page
                    j, r = lo // BLOCK, int(self.offsets[i]) + a - p
                    rows, off = x[r:r + b - a], slack[r:r + b - a]
                    most = rows.abs().amax((0, 2))
                    s = scale_of(most)
                    # a largest element within the arithmetic of a border may fall on either side
                    near = (scale_of(most - off.amax((0, 2))) != s) | (scale_of(most + off.amax((0, 2))) != s)
                    if a % BLOCK:
                        old = scales[at, :, j].double()
                        s = torch.maximum(s, old)
                        near &= gscale[at, :, j] > old
                        older = slice(j * BLOCK, lo)
                    s = torch.where(near, gscale[at, :, j].double(), s)
                    if a % BLOCK:
                        ratio = (old / s)[:, None, None]
                        e = e4m3(want_n[at, :, older] * ratio)
                        want_n[at, :, older] = torch.where(ratio < 1, e, want_n[at, :, older])
                    want_s[at, :, j] = s
                    y = rows.transpose(0, 1) / s[:, None, None]
                    want_n[at, :, lo:lo + b - a] = y
                    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
                    d = off.transpose(0, 1) / s[:, None, None]
                    # (a value a little below a power of two may be rounded with the wider step)
                    tol[at, :, lo:lo + b - a] = step / 2 * (1 + 2.0 ** -20) + 2 * d
                    a = b
            assert torch.equal(gscale.double(), want_s), f"scales of {'kv'[kind]}"
            within(got.float(), want_n, tol, f"numbers of {'kv'[kind]}")
        return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,p", [([1], [0]), ([1, 1, 1, 1], [0, 15, 16, 1001]), ([40, 0, 1, 17], [3, 9, 64, 31]),
                                 ([0, 700, 3, 1, 130], [5, 20, 47, 11, 64])])
@pytest.mark.parametrize("H,Hkv,D,page,rot,il", [(4, 2, 64, 16, 64, False), (14, 2, 64, 32, 16, True),
                                                 (40, 8, 128, 64, 128, False), (3, 3, 128, 256, 120, False),
                                                 (8, 1, 64, 16, 2, False), (5, 1, 128, 32, 0, False),
                                                 (6, 2, 64, 64, 50, True), (4, 1, 64, 16, 50, False)])
def test_matches_definition(dtype, n, p, H, Hkv, D, page, rot, il):
    Append(n, p, H, Hkv, D, dtype, page, rot, il, seed=H + rot + len(n)).check()


def test_many_short_sequences_and_tail_rows():
    rng = np.random.default_rng(3)
    n, p = rng.integers(0, 40, 150).tolist(), rng.integers(0, 3000, 150).tolist()
    Append(n, p, 8, 2, 64, "bf16", 32, seed=4, tail_rows=5).check()
    Append([1] * 700, rng.integers(0, 500, 700).tolist(), 4, 2, 64, "f16", 16, seed=5).check()


def test_far_positions_and_scale():
    Append([33, 1], [131000, 2000000], 8, 2, 128, "bf16", 64, seed=6, scale=1.25).check()


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 30])
def test_sizes_of_rows(size):
    Append([20, 1], [5, 9], 4, 2, 64, "f32", 16, seed=7, size=size).check()


def test_zero_rows_and_scales_that_were_never_written():
    """Rows of zeros have the least scale; a scale of 0 (fresh memory) is what any row grows."""
    a = Append([1, 16], [3, 16], 4, 2, 64, "bf16", 16, seed=8)
    for t in (a.k, a.v):
        t.zero_()
    for s in a.scales:
        s.zero_()
    before = [x.clone() for x in a.pages]
    a.run()
    for kind in range(2):
        block = int(a.table[0, 0])
        assert (a.scales[kind][block] == 2.0 ** -60).all()
        assert (a.pages[kind][block, :, :4].float() == 0).all()  # (the older ones stood for 0)
        assert torch.equal(a.pages[kind][block, :, 4:].view(torch.uint8), before[kind][block, :, 4:].view(torch.uint8))
        full = int(a.table[1, 1])
        assert (a.pages[kind][full].float() == 0).all() and (a.scales[kind][full] == 2.0 ** -60).all()


def test_largest_on_the_border_of_a_scale():
    """448 2^k is the largest that scale 2^k holds; the next number takes 2^(k + 1)."""
    a = Append([1, 1], [0, 0], 1, 1, 64, "f32", 16, rot=0, seed=9)
    for r, most in enumerate((448.0 * 2.0 ** -5, float(np.nextafter(np.float32(448.0 * 2.0 ** -5), np.float32(1e9))))):
        a.v[r].fill_(0.001)
        a.v[r, 0, 17] = -most
    a.run()
    assert a.scales[1][int(a.table[0, 0]), 0, 0] == 2.0 ** -5
    assert a.scales[1][int(a.table[1, 0]), 0, 0] == 2.0 ** -4
    assert a.pages[1][int(a.table[0, 0]), 0, 0, 17].float() == -448
    assert a.pages[1][int(a.table[1, 0]), 0, 0, 17].float() == -224


def test_one_by_one_or_together():
    """The scales are the same however the rows came; the numbers stand for the same values down to
    the rounding of the least ones."""
    n = 50
    together = Append([n], [0], 4, 2, 64, "bf16", 64, seed=10)
    alone = Append([n], [0], 4, 2, 64, "bf16", 64, seed=10)
    together.run()
    cache = alone.cache()
    for t in range(n):
        alone.positions.fill_(t)
        offsets = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        b = B.PagedBatch(alone.positions, offsets, alone.page_table, 1, 1)
        out = torch.empty(1, 4, 64, dtype=torch.bfloat16, device=DEV)
        B.kvs_rope_scatter_paged_q8(alone.q[t:t + 1], alone.k[t:t + 1], alone.v[t:t + 1], out, cache, b,
                                    alone.inv_freq, d_status=alone.status)
    at = int(together.table[0, 0])
    for kind in range(2):
        assert torch.equal(together.scales[kind][at, :, :4], alone.scales[kind][at, :, :4])
        x, y = together.pages[kind][at, :, :n].float(), alone.pages[kind][at, :, :n].float()
        # a number of 2^-6 or more is exact under every growth; one below was rounded to 2^-9 under
        # an earlier scale's finer steps first: half a step more
        assert ((x - y).abs() <= torch.where(x.abs() >= 2.0 ** -6, 0.0, 2.0 ** -9)).all()


def test_in_place_and_bad_input():
    a = Append([3, 20, 1], [14, 3, 100], 8, 2, 64, "bf16", 16, seed=11)
    q = a.q.clone()
    want = a.run()
    a.run(q_out=a.q)
    assert torch.equal(a.q, want)
    a.q.copy_(q)
    a.positions[1] = -3
    pages, scales = [x.clone() for x in a.pages], [x.clone() for x in a.scales]
    out = a.run()
    assert int(a.status.item()) == B.KVS_ERR_POSITION
    assert torch.isnan(out[3:23]).all() and torch.equal(out[:3], want[:3]) and torch.equal(out[23:], want[23:])
    a.positions[1] = 3
    a.status.zero_()
    a.page_table[1, 1] = 1 << 20
    out = a.run()
    assert int(a.status.item()) == B.KVS_ERR_PAGE
    assert torch.equal(out, want)
    for x, y in zip(a.pages + a.scales, pages + scales):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_captured_call():
    a = Append([1] * 6, [0, 5, 16, 31, 200, 77], 8, 2, 128, "bf16", 32, seed=13)
    out = a.run()
    first = out.clone()
    cache = a.cache()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.kvs_rope_scatter_paged_q8(a.q, a.k, a.v, out, cache, a.batch, a.inv_freq)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("dtype", DTYPES)
def test_from_rows_to_a_token(dtype):
    """A prompt and decode steps through the cache: scatter, attention, and a token drawn from what
    stands for logits, against the same in 64 bits on the values that the cache holds."""
    H, Hkv, D, page, steps = 8, 2, 64, 16, 5
    n0 = [37, 5]
    total = [a + steps for a in n0]
    g = torch.Generator(device=DEV)
    g.manual_seed(14)
    T = DTYPES[dtype]
    rows = [torch.empty(t, (H + 2 * Hkv) * D, device=DEV).normal_(generator=g).to(T) for t in total]
    pages = [torch.zeros(8, Hkv, page, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    scales = [torch.zeros(8, Hkv, page // BLOCK, device=DEV) for _ in range(2)]
    cache = B.PagedCacheQ8(pages[0], pages[1], scales[0], scales[1])
    table = torch.tensor([[3, 1, 6], [0, 7, -1]], dtype=torch.int32, device=DEV)
    inv = torch.from_numpy((10000.0 ** (-np.arange(D // 2) * 2.0 / D)).astype(np.float32)).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    weight = torch.empty(H * D, 500, device=DEV).normal_(generator=g)
    done = [0, 0]
    for n in [n0] + [[1, 1]] * steps:
        qkv = torch.cat([r[a:a + b] for r, a, b in zip(rows, done, n)])
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((H * D, Hkv * D, Hkv * D), 1))
        batch = B.PagedBatch(torch.tensor(done, dtype=torch.int32, device=DEV),
                             torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV), table, sum(n), max(n))
        turned, out = torch.empty_like(q.contiguous()), torch.empty(sum(n), H, D, dtype=T, device=DEV)
        B.kvs_rope_scatter_paged_q8(q, k, v, turned, cache, batch, inv, d_status=status)
        B.kvs_paged_attention_q8(turned, cache, batch, out, d_status=status,
                                 workspace=B.paged_attention_q8_workspace(cache, batch, H))
        done = [a + b for a, b in zip(done, n)]
        at = 0
        for i in range(2):
            use = table[i, :-(-done[i] // page)].tolist()
            kk, vv = ((x[use].double() * s[use].double().repeat_interleave(BLOCK, 2)[..., None])
                      .transpose(0, 1).reshape(Hkv, -1, D)[:, :done[i]] for x, s in zip(pages, scales))
            qq = turned[at:at + n[i]].double().view(n[i], Hkv, H // Hkv, D)
            z = torch.einsum("tged,gld->gtel", qq, kk) / math.sqrt(D)
            far = torch.arange(done[i], device=DEV)[None] > (done[i] - n[i] + torch.arange(n[i], device=DEV))[:, None]
            w = torch.softmax(z.masked_fill(far[None, :, None], -math.inf), -1)
            ref = torch.einsum("gtel,gld->tged", w, vv).reshape(n[i], H, D)
            # float16 weights 2^-12, a rounding to the type, scores and sums under 2^-16
            tol = (2.0 ** -11 + half_step(T)) * vv.abs().amax() + 2.0 ** -16
            within(out[at:at + n[i]], ref, tol.expand_as(ref), f"{i} at {done[i]}")
            at += n[i]
    assert int(status.item()) == 0
    last = out[[n[0] - 1, sum(n) - 1]].float().flatten(1) @ weight
    u = torch.tensor([0.3, 0.8], device=DEV)
    got = B.kvs_sample_logits(last, u, top_k=torch.full((2,), 1, dtype=torch.int32, device=DEV))
    assert torch.equal(got.long(), last.argmax(1))
