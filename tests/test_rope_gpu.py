"""kvs_rope_scatter_paged against the definition in 64 bits, and the pages it writes."""
import math

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, Paged, half_step, least_step, within
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


def rotate64(x, pos, inv_freq, interleaved, scale):
    """x [rows, heads, D] rotated, with the bound of the kernel's arithmetic."""
    x = x.double()
    half = inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()
    c, s = (scale * f(angle)[:, None] for f in (torch.cos, torch.sin))
    out, size = x.clone(), x.abs()
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = a.abs() + b.abs()
    return out, size


def make_case(n, p, H, Hkv, D, dtype, page, seed, tail_rows=0):
    b = Paged(n, p, H, Hkv, D, dtype, page, seed=seed, tail_rows=tail_rows)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1)
    b.new_k, b.new_v = (torch.empty(b.rows, Hkv, D, device=DEV).normal_(generator=g).to(b.dtype)
                        for _ in range(2))
    return b


def check(b, q_out, inv_freq, interleaved, scale, k0, v0, q=None):
    """q_out, the rows written and every other row of the pages (as they were: k0, v0)."""
    live = sum(b.n)
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(b.n, b.p)]).to(DEV)
    u = half_step(b.dtype)
    # cos and sin: the angle to 2^-25 half turns (pi 2^-25), sincospi to 2 units of 2^-24, the
    # product with scale 2^-24, two products and a sum 3 x 2^-24: under 2^-21 of |a| + |b|;
    # then one rounding to the type, u of the result or, below the normal range, its least step
    def close(got, ref):
        ref, size = ref
        within(got, ref, abs(scale) * size * 2.0 ** -21 + u * ref.abs() * 1.01 + least_step(b.dtype))
    turned = rotate64(b.q[:live] if q is None else q[:live], pos, inv_freq, interleaved, scale)
    close(q_out[:live], turned)
    rest = 2 * inv_freq.numel()
    src = (b.q if q is None else q)[:live]
    assert torch.equal(q_out[:live, :, rest:], src[:, :, rest:])  # copied, to the bit
    want_k, size_k = rotate64(b.new_k[:live], pos, inv_freq, interleaved, scale)
    seq = torch.repeat_interleave(torch.arange(len(b.n)), torch.tensor(b.n)).to(DEV)
    page = b.page_table[seq, pos // b.page].long()
    slot = pos % b.page
    close(b.k_pages[page, :, slot], (want_k, size_k))
    assert torch.equal(b.v_pages[page, :, slot], b.new_v[:live])
    k1, v1 = b.k_pages.clone(), b.v_pages.clone()
    k1[page, :, slot], v1[page, :, slot] = k0[page, :, slot], v0[page, :, slot]
    as_int = torch.int32 if b.dtype == torch.float32 else torch.int16
    assert torch.equal(k1.view(as_int), k0.view(as_int)), "another row of K was written"
    assert torch.equal(v1.view(as_int), v0.view(as_int)), "another row of V was written"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,D,rot", [(4, 2, 64, 64), (14, 2, 64, 16), (40, 8, 128, 128),
                                         (8, 1, 128, 64), (3, 3, 64, 2), (6, 2, 128, 90),
                                         (6, 2, 64, 56), (5, 1, 64, 0), (16, 2, 128, 120)])
def test_matches_definition(dtype, interleaved, H, Hkv, D, rot):
    b = make_case([1, 37, 0, 5, 1], [0, 11, 4, 1000, 2047], H, Hkv, D, dtype, 16, seed=rot + H, tail_rows=2)
    inv, scale = (B.kvs_rope_frequencies(rot) if rot else (torch.empty(0, device=DEV), 1.0))
    k0, v0 = b.k_pages.clone(), b.v_pages.clone()
    out = torch.full_like(b.q, 7.0)
    B.kvs_rope_scatter_paged(b.q, b.new_k, b.new_v, out, b.cache, b.batch, inv, interleaved=interleaved,
                             scale=1.25, d_status=b.status)
    assert int(b.status.item()) == 0
    check(b, out, inv, interleaved, 1.25, k0, v0)
    assert (out[sum(b.n):] == 7).all(), "wrote behind the last sequence"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_positions(dtype):
    """Angles of many turns keep full precision (positions to 2^31 over a shared first page)."""
    n, D, Hkv = [3, 1, 1], 64, 2
    b = make_case([1], [0], 4, Hkv, D, dtype, 16, seed=1)
    p = [131070, 1 << 24, (1 << 30) + 12345]
    k = torch.zeros(2, Hkv, 16, D, dtype=b.dtype, device=DEV)
    b.n, b.p, b.rows, b.page = n, p, 5, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    b.q = torch.empty(5, 4, D, device=DEV).normal_(generator=g).to(b.dtype)
    b.new_k = torch.zeros(5, Hkv, D, dtype=b.dtype, device=DEV)
    max_pages = (max(p) + 1) // 16 + 1
    table = torch.zeros(3, max_pages, dtype=torch.int32, device=DEV)  # all page 0: only q is looked at
    batch = B.PagedBatch(torch.tensor(p, dtype=torch.int32, device=DEV),
                         torch.tensor([0, 3, 4, 5], dtype=torch.int32, device=DEV), table, 5, 3)
    inv, scale = B.kvs_rope_frequencies(64, base=500000.0)
    out = torch.empty_like(b.q)
    B.kvs_rope_scatter_paged(b.q, b.new_k, b.new_k, out, B.PagedCache(k, k.clone()), batch, inv,
                             d_status=b.status)
    assert int(b.status.item()) == 0
    pos = torch.cat([torch.arange(a, a + c) for a, c in zip(p, n)]).to(DEV)
    ref, size = rotate64(b.q, pos, inv, False, 1.0)
    # 1 / 2 pi in double: 2^-53 of the turns, so 2^-53 p w / 2 pi turns more
    slack = 2.0 ** -53 * pos.double()[:, None, None] * 2 * math.pi
    within(out, ref, size * (2.0 ** -21 + slack) + half_step(b.dtype) * ref.abs() * 1.01 + least_step(b.dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_column_blocks_and_in_place(dtype):
    H, Hkv, D = 8, 2, 64
    b = make_case([20, 1], [100, 7], H, Hkv, D, dtype, 32, seed=3)
    qkv = torch.cat([b.q.flatten(1), b.new_k.flatten(1), b.new_v.flatten(1)], 1)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, Hkv * D, Hkv * D], 1))
    before = q.clone()
    inv, scale = B.kvs_rope_frequencies(D)
    k0, v0 = b.k_pages.clone(), b.v_pages.clone()
    B.kvs_rope_scatter_paged(q, k, v, q, b.cache, b.batch, inv, d_status=b.status)
    assert int(b.status.item()) == 0
    check(b, q, inv, False, scale, k0, v0, q=before)
    assert torch.equal(k, b.new_k) and torch.equal(v, b.new_v)


def test_bad_input_is_reported_and_skipped():
    inv, _ = B.kvs_rope_frequencies(64)
    for what, code in (("page", B.KVS_ERR_PAGE), ("position", B.KVS_ERR_POSITION), ("rows", B.KVS_ERR_ROWS)):
        b = make_case([2, 3, 1], [30, 20, 10], 4, 2, 64, "f16", 16, seed=4)
        if what == "page":
            b.page_table[1, 1] = 10 ** 6
        elif what == "position":
            b.positions[1] = -1
        else:
            b.row_offsets[3] = 99
        k0 = b.k_pages.clone()
        out = torch.full_like(b.q, 7.0)
        B.kvs_rope_scatter_paged(b.q, b.new_k, b.new_v, out, b.cache, b.batch, inv, d_status=b.status)
        assert int(b.status.item()) == code, what
        changed = (k0.view(torch.int16) != b.k_pages.view(torch.int16)).any(-1).any(1)  # [pages, slots]
        written = {"page": 3, "position": 3, "rows": 5}[what]
        assert int(changed.sum()) == written, what
        assert out[2:5].isnan().all() == (what == "position")
        if what == "rows":
            assert (out[5:] == 7).all()


@pytest.mark.parametrize("kind", range(5))
def test_length_scaling_rules_reach_the_kernel(kind):
    b = make_case([9], [4090], 4, 2, 64, "f32", 16, seed=5)
    inv, scale = B.kvs_rope_frequencies(64, kind=kind, factor=4.0, original_len=1024.0)
    k0, v0 = b.k_pages.clone(), b.v_pages.clone()
    out = torch.empty_like(b.q)
    B.kvs_rope_scatter_paged(b.q, b.new_k, b.new_v, out, b.cache, b.batch, inv, scale=scale, d_status=b.status)
    check(b, out, inv, False, scale, k0, v0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_serving_iteration(dtype):
    """Rotary scatter, attention and token choice together, captured once and replayed: a prompt
    chunk, then decode steps, against the same steps in 64 bits."""
    H, Hkv, D, page, V = 8, 2, 64, 16, 500
    dt = DTYPES[dtype]
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    M, chunk, steps = 3, [40, 1, 17], 4
    start = [0, 0, 0]
    k_pages = torch.full((40, Hkv, page, D), math.nan, dtype=dt, device=DEV)
    v_pages = torch.full_like(k_pages, math.nan)
    table = torch.randperm(39, generator=g, device=DEV)[:24].view(3, 8).to(torch.int32)
    positions = torch.zeros(M, dtype=torch.int32, device=DEV)
    offsets = torch.zeros(M + 1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = B.PagedCache(k_pages, v_pages)
    inv, scale = B.kvs_rope_frequencies(D)
    head = torch.empty(V, H * D, device=DEV).normal_(generator=g) / 16
    kr, vr = [[torch.empty(0, Hkv, D, dtype=torch.float64, device=DEV) for _ in range(M)] for _ in range(2)]
    history = torch.randint(0, V, (M * 12,), generator=g, device=DEV).to(torch.int32)
    hist_off = torch.arange(0, 12 * M + 1, 12, device=DEV, dtype=torch.int32)
    rep = torch.full((M,), 1.3, device=DEV)
    u = half_step(dt)

    def step(n, captured):
        rows = sum(n)
        x = torch.empty(rows, (H + 2 * Hkv) * D, device=DEV).normal_(generator=g).to(dt)
        captured["x"].copy_(x)
        offsets.copy_(torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32))
        captured["run"]()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        # the same in 64 bits, from the rotated rows as the type holds them
        at = 0
        for i in range(M):
            p = int(positions[i])
            pos = torch.arange(p, p + n[i], device=DEV)
            q, k, v = (t.unflatten(1, (-1, D)) for t in x[at:at + n[i]].split([H * D, Hkv * D, Hkv * D], 1))
            q, k = (rotate64(t, pos, inv, False, scale)[0].to(dt).double() for t in (q, k))
            kr[i], vr[i] = torch.cat([kr[i], k]), torch.cat([vr[i], v.double()])
            s = torch.einsum("tged,lgd->gtel", q.view(n[i], Hkv, H // Hkv, D), kr[i]) / math.sqrt(D)
            far = torch.arange(len(kr[i]), device=DEV)[None] > pos[:, None]
            w = torch.softmax(s.masked_fill(far[None, :, None], -math.inf), -1)
            o = torch.einsum("gtel,lgd->tged", w, vr[i]).reshape(n[i], H, D)
            got = captured["out"][at:at + n[i]].double()
            # the rotated rows may round to the neighbour (a step, 2 u): scores off by 4 u |s|, and
            # the attention's own bound: u |v| for the weights, u |o| for the result
            vm, sm = vr[i].abs().max(), torch.einsum("tgd,lgd->gtl", q.view(n[i], Hkv, -1, D).abs().amax(2), kr[i].abs()).max() / math.sqrt(D)
            within(got, o, (vm * (8 * u * sm + 4 * u + 2.0 ** -16)).expand_as(o))
            at += n[i]
        ids = captured["ids"].cpu().numpy()
        y = captured["logits"].cpu().numpy()
        assert [int(np.argmax(r)) for r in y] == ids.tolist()
        positions.add_(torch.tensor(n, dtype=torch.int32, device=DEV))

    def make(n):
        rows = sum(n)
        c = dict(x=torch.zeros(rows, (H + 2 * Hkv) * D, dtype=dt, device=DEV),
                 out=torch.zeros(rows, H, D, dtype=dt, device=DEV), logits=torch.zeros(M, V, device=DEV),
                 ids=torch.zeros(M, dtype=torch.int32, device=DEV))
        batch = B.PagedBatch(positions, offsets, table, rows, max(n))
        ws = B.paged_attention_workspace(cache, batch, H)
        last = torch.tensor(np.cumsum(n) - 1, device=DEV)

        def run():
            q, k, v = (t.unflatten(1, (-1, D)) for t in c["x"].split([H * D, Hkv * D, Hkv * D], 1))
            B.kvs_rope_scatter_paged(q, k, v, q, cache, batch, inv, scale=scale, d_status=status)
            B.kvs_paged_attention(q, cache, batch, c["out"], workspace=ws, d_status=status)
            c["logits"].copy_(c["out"][last].float().flatten(1) @ head.T)
            B.kvs_process_logits(c["logits"], c["logits"], token_ids=c["ids"], history=history,
                                 history_offsets=hist_off, repetition=rep, d_status=status)
        c["run"] = run
        return c

    step(chunk, make(chunk))
    c = make([1] * M)
    offsets.copy_(torch.arange(M + 1, dtype=torch.int32))
    saved = k_pages.clone(), v_pages.clone()
    c["run"]()  # set-up before the capture (its rows are written again by the first step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c["run"]()
    k_pages.copy_(saved[0])
    v_pages.copy_(saved[1])
    c["kept"] = c["run"]  # the graph uses the tensors that this closure holds
    c["run"] = graph.replay
    for _ in range(steps):
        step([1] * M, c)
