"""The 8-bit cache's entry points and the choice of a token where a program meets them unprepared:
first calls inside a capture, waits that run out, shared pages, one workspace in turn, two threads,
large pools and batches."""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, within
from q8_helpers import BLOCK, E4M3, PagedQ8, scale_of
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


# every kernel: decode steps by clusters and by ranges, of few and more rows, chunks in 16 and 32 bits
KINDS = {
    "clusters": dict(n=[1, 1], p=[300, 5], H=8, Hkv=2, D=64, dtype="f16", page=16),
    "ranges": dict(n=[1, 1], p=[9000, 5000], H=8, Hkv=2, D=128, dtype="bf16", page=64, columns=2 ** 14),
    "ranges f32": dict(n=[1, 1], p=[9000, 5000], H=8, Hkv=2, D=64, dtype="f32", page=64, columns=2 ** 14),
    "few rows more": dict(n=[3, 1], p=[9000, 500], H=8, Hkv=2, D=64, dtype="f16", page=64, columns=2 ** 14),
    "chunks": dict(n=[170, 1, 40], p=[3, 900, 2000], H=8, Hkv=2, D=128, dtype="bf16", page=32),
    "chunks f16": dict(n=[170, 1, 40], p=[3, 900, 2000], H=14, Hkv=2, D=64, dtype="f16", page=16),
    "short f32": dict(n=[20, 1], p=[3, 900], H=8, Hkv=2, D=128, dtype="f32", page=32),
    "long f32": dict(n=[300, 1, 40], p=[3, 900, 2000], H=8, Hkv=2, D=64, dtype="f32", page=32),
    "long f32 wide": dict(n=[120, 50], p=[300, 900], H=20, Hkv=4, D=128, dtype="f32", page=32),
}


def kind(name, seed=0, **kw):
    return PagedQ8(**dict(KINDS[name], seed=seed, **kw))


@pytest.mark.parametrize("name", KINDS)
def test_every_kernel(name):
    b = kind(name, seed=1, tail_rows=3)
    out = b.attend()
    b.check(out)
    assert (out[sum(b.n):] == 7).all()
    again = b.attend()
    assert torch.equal(out, again)


@pytest.mark.parametrize("n", [127, 128, 129, 200, 224, 225])
@pytest.mark.parametrize("p", [0, 1, 62, 63, 64, 511])
def test_tile_edges_of_long_float32_chunks(n, p):
    PagedQ8([n], [p], 14, 2, 64, "f32", 16, seed=n + p).check(
        PagedQ8([n], [p], 14, 2, 64, "f32", 16, seed=n + p).attend())


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from paged_helpers import DEV
from test_q8_edges_gpu import KINDS, kind
from test_rope_q8_gpu import Append
from split_flash_decoding_kvcachescatter_gb300 import binding as B
kinds = [kind(name) for name in KINDS]
a, part = Append([5, 1], [3, 16], 8, 2, 64, "bf16", 16), Append([5, 1], [3, 16], 8, 2, 64, "f32", 16, rot=24)
x = torch.randn(3, 1000, device=DEV)
ids, u = torch.empty(3, dtype=torch.int32, device=DEV), torch.full((3,), 0.5, device=DEV)
one = torch.ones(3, dtype=torch.int32, device=DEV)
outs = [torch.zeros_like(b.q) for b in kinds]
turned = [torch.zeros_like(r.q.contiguous()) for r in (a, part)]
caches = [r.cache() for r in (a, part)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for b, out in zip(kinds, outs):
        b.attend(out=out)
    for r, to, cache in zip((a, part), turned, caches):
        B.kvs_rope_scatter_paged_q8(r.q, r.k, r.v, to, cache, r.batch, r.inv_freq, d_status=r.status)
    B.kvs_sample_logits(x, u, token_ids=ids, top_k=one)
graph.replay()
torch.cuda.synchronize()
for b, out in zip(kinds, outs):
    b.check(out)
assert torch.equal(ids.long(), x.argmax(1)) and all(t.abs().sum() > 0 for t in turned)
assert int(a.status.item()) == int(part.status.item()) == 0
print("fine")
"""


def test_first_calls_of_a_process_inside_a_capture():
    code = FIRST_CALL.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("name", KINDS)
def test_waits_that_run_out_are_reported(name):
    """With the wait bound at zero some wait of some block runs out: the status says so, rows behind
    the last sequence stay, and the same workspace serves the next call."""
    b = kind(name, seed=17, tail_rows=2)
    prev = B.kvs_set_wait_limit_ns(0)
    try:
        out = b.attend()
        torch.cuda.synchronize()
        assert int(b.status.item()) == B.KVS_ERR_TIMEOUT
        assert (out[sum(b.n):] == 7).all()
    finally:
        B.kvs_set_wait_limit_ns(prev)
    b.status.zero_()
    b.check(b.attend())


@pytest.mark.parametrize("limit", [300, 3000, 30000])
def test_waits_that_run_out_anywhere(limit):
    for name in ("ranges", "chunks", "long f32"):
        b = kind(name, seed=18)
        prev = B.kvs_set_wait_limit_ns(limit)
        try:
            b.attend()
            torch.cuda.synchronize()
            assert int(b.status.item()) in (B.KVS_OK, B.KVS_ERR_TIMEOUT)
        finally:
            B.kvs_set_wait_limit_ns(prev)
        b.status.zero_()
        b.check(b.attend(), name)


def test_one_workspace_for_every_kernel_and_their_graphs():
    kinds = [kind(name, seed=5) for name in KINDS]
    ws = max((b.workspace for b in kinds), key=lambda t: t.numel())
    outs = [torch.zeros_like(b.q) for b in kinds]
    graphs = []
    for b, out in zip(kinds, outs):
        b.workspace = ws
        b.attend(out=out)
    torch.cuda.synchronize()
    for b, out in zip(kinds, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            b.attend(out=out)
    order = list(range(len(kinds)))
    for order in (order, order[::-1], order[::2] * 2):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
            kinds[order[0]].attend()
        torch.cuda.synchronize()
        for i in order:
            kinds[i].check(outs[i], f"order {order}, {i}")


def test_two_threads():
    cases = [kind("ranges", seed=9), kind("chunks", seed=10), kind("long f32", seed=11)]
    outs, streams, errors = [torch.zeros_like(b.q) for b in cases], [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()

    def work(i):
        try:
            for _ in range(30):
                cases[i].attend(out=outs[i], stream=streams[i])
        except Exception as e:  # told to the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for b, out in zip(cases, outs):
        b.check(out)


@pytest.mark.parametrize("name,shared", [("clusters", 5), ("chunks", 3), ("long f32", 2)])
def test_sequences_share_the_pages_of_a_prefix(name, shared):
    c = KINDS[name]
    b = kind(name, seed=4, n=[c["n"][0], 1, 2][:3], p=[200, 190, 210])
    for i in (1, 2):
        b.page_table[i, :shared] = b.page_table[0, :shared]
        for mine in (b.k, b.v):
            mine[i][:, :shared * b.page] = mine[0][:, :shared * b.page]
    b.check(b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("max_new", [17, 500, 2 ** 20])
def test_bound_on_new_tokens_above_all(dtype, max_new):
    """A program that always passes the largest chunk: decode steps then take the chunk kernels."""
    b = PagedQ8([1, 1, 2, 0, 1], [700, 0, 31, 2, 4000], 8, 2, 64, dtype, 32, seed=3)
    b.batch = B.PagedBatch(b.positions, b.row_offsets, b.page_table, b.rows, max_new)
    b.workspace = B.paged_attention_q8_workspace(b.cache, b.batch, 8)
    out = b.attend()
    ref, bound = b.reference()
    # (single tokens by the chunk kernels: weights rounded to float16, 2^-11 of the values' size)
    v = max(float(x.abs().max()) for x in b.v if x.numel())
    within(out, ref, bound + (0 if dtype == "f32" else 2.0 ** -11 * v + 2.0 ** -20 * v))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,D", [(12, 2, 64), (4, 1, 128), (512, 64, 64), (31, 31, 64)])
@pytest.mark.parametrize("n,p", [([1, 1, 0, 1], [70, 0, 3, 400]), ([30, 1, 0, 100], [70, 0, 3, 40])])
def test_other_head_layouts(dtype, H, Hkv, D, n, p):
    b = PagedQ8(n, p, H, Hkv, D, dtype, 16, seed=H + D)
    b.check(b.attend())


@pytest.mark.parametrize("dtype,n", [("f16", 1), ("f32", 1), ("bf16", 40), ("f32", 300)])
def test_most_sequences_of_a_batch_are_empty(dtype, n):
    """The largest number of sequences, all but the first and the last without a token."""
    M = 2 ** 20
    b = PagedQ8([n, 1], [700, 90], 8, 2, 64, dtype, 16, seed=13)
    wide = torch.zeros(M, b.page_table.shape[1], dtype=torch.int32, device=DEV)
    wide[0], wide[-1] = b.page_table[0], b.page_table[1]
    offsets = torch.full((M + 1,), n, dtype=torch.int32, device=DEV)
    offsets[0], offsets[-1] = 0, n + 1
    positions = torch.zeros(M, dtype=torch.int32, device=DEV)
    positions[0], positions[-1] = 700, 90
    b.batch = B.PagedBatch(positions, offsets, wide, n + 1, n)
    b.check(b.attend())


@pytest.mark.parametrize("n", [1, 60])
def test_pages_past_32_bit_offsets(n):
    """A pool of 5 GB: pages at its end, read and written."""
    D, page = 128, 2 ** 15
    pages = -(-5 * 2 ** 30 // (page * D))
    kp, vp = (torch.zeros(pages, 1, page, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    ks, vs = (torch.ones(pages, 1, page // BLOCK, device=DEV) for _ in range(2))
    b = PagedQ8([n], [50], 4, 1, D, "bf16", 128, seed=3)
    at = int(b.table_host[0, 0])
    L = 50 + n
    for big, small in ((kp, b.k_pages), (vp, b.v_pages)):
        big.view(torch.uint8)[pages - 1, 0, :L] = small.view(torch.uint8)[at, 0, :L]
    for big, small in ((ks, b.k_scales), (vs, b.v_scales)):
        big[pages - 1, 0, :-(-L // BLOCK)] = small[at, 0, :-(-L // BLOCK)]
    b.cache = B.PagedCacheQ8(kp, vp, ks, vs)
    table = torch.full((1, 2), pages - 1, dtype=torch.int32, device=DEV)
    b.batch = B.PagedBatch(b.positions, b.row_offsets, table, n, n)
    b.check(b.attend())
    # the rows appended there: what is read back is within a step of them, other pages stay
    new = torch.ones(n, 1, D, dtype=torch.bfloat16, device=DEV) * 0.75
    inv = torch.zeros(D // 2, device=DEV)
    out = torch.empty_like(b.q)
    B.kvs_rope_scatter_paged_q8(b.q, new, new, out, b.cache, b.batch, inv, d_status=b.status)
    assert int(b.status.item()) == 0 and torch.equal(out, b.q)  # (an angle of zero)
    for pool, scales in ((kp, ks), (vp, vs)):
        got = pool[pages - 1, 0, 50:L].float() * scales[pages - 1, 0].repeat_interleave(BLOCK)[50:L, None]
        # (the first of them may share a block, and a larger scale, with older rows)
        # (half a step: 2^-4 of it, or 2^-10 of the scale)
        within(got, torch.full_like(got, 0.75).double(),
               (0.75 * 2.0 ** -4 + scales[pages - 1, 0].max().double() * 2.0 ** -10).expand_as(got))
        assert not pool[:8].view(torch.uint8).any() and not pool[pages - 1, 0, L:].view(torch.uint8).any()


def test_more_appended_rows_than_32_bit_thread_numbers():
    """2^24 rows: every sequence's rows are found and written."""
    N, D, page = 2 ** 24 + 300, 64, 2 ** 15
    n, p = [N - 257, 0, 256, 1], [0, 5, 3, 2 ** 20]
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    qkv = torch.empty(N, 3 * D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    q, k, v = (qkv[:, j * D:(j + 1) * D].unflatten(1, (1, D)) for j in range(3))
    pages = -(-n[0] // page)
    pool = [torch.zeros(pages + 2, 1, page, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    scales = [torch.zeros(pages + 2, 1, page // BLOCK, device=DEV) for _ in range(2)]
    cache = B.PagedCacheQ8(pool[0], pool[1], scales[0], scales[1])
    table = torch.zeros(4, pages, dtype=torch.int32, device=DEV)
    table[0] = torch.arange(pages, dtype=torch.int32, device=DEV)
    table[2], table[3] = pages, pages + 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    batch = B.PagedBatch(i32(p), i32(np.concatenate([[0], np.cumsum(n)])), table, N, max(n))
    status, inv = i32([0]), torch.zeros(D // 2, device=DEV)  # (angles of zero: rows as they are)
    out = torch.zeros(N, 1, D, dtype=torch.bfloat16, device=DEV)
    B.kvs_rope_scatter_paged_q8(q, k, v, out, cache, batch, inv, d_status=status)
    assert int(status.item()) == 0
    assert torch.equal(out, q)
    for x, numbers, s in ((k, pool[0], scales[0]), (v, pool[1], scales[1])):
        for page_at, row, first, count in ((0, 0, 0, 4096), (pages - 1, (pages - 1) * page, 0, n[0] - (pages - 1) * page),
                                           (pages, n[0], 3, 256), (pages + 1, N - 1, 2 ** 20 % page, 1)):
            want = x[row:row + count, 0].double()
            blocks = torch.arange(first, first + count, device=DEV) // BLOCK
            got_s = s[page_at, 0][blocks].double()
            most = torch.zeros(page // BLOCK, dtype=torch.float64, device=DEV)
            most.scatter_reduce_(0, blocks, want.abs().amax(1), "amax")
            assert torch.equal(got_s, scale_of(most)[blocks])
            got = numbers[page_at, 0, first:first + count].double() * got_s[:, None]
            # half a step of e4m3: 2^-4 of a number, 2^-10 under the scale
            within(got, want, want.abs() * 2.0 ** -4 * 1.001 + got_s[:, None] * 2.0 ** -10)


def test_without_a_status_word():
    b = PagedQ8([1, 20], [30, 0], 8, 2, 64, "f16", 16, seed=11)
    out = torch.full_like(b.q, 7.0)
    B.kvs_paged_attention_q8(b.q, b.cache, b.batch, out, workspace=b.workspace)
    b.check(out)
    b.page_table[0, 0] = -1
    B.kvs_paged_attention_q8(b.q, b.cache, b.batch, out, workspace=b.workspace)
    assert out[0].isnan().all() and not out[1:].isnan().any()


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_bad_pages_of_float32_chunks(n, D):
    b = PagedQ8([n, n], [40, 100], 8, 2, D, "f32", 16, seed=6)
    good, bound = b.reference()
    b.page_table[0, 1] = 1 << 20
    out = b.attend()
    assert int(b.status.item()) == B.KVS_ERR_PAGE
    assert torch.isnan(out[:n]).all()
    within(out[n:], good[n:], bound[n:], "beside a bad page")
    b.positions[0] = 1 << 20
    b.status.zero_()
    out = b.attend()
    assert int(b.status.item()) == B.KVS_ERR_POSITION
    assert torch.isnan(out[:n]).all()
    within(out[n:], good[n:], bound[n:], "beside a bad position")


def test_append_and_attention_of_a_step_in_one_graph():
    """A layer's step captured once: each replay appends at the positions of its time and reads
    them back, on a stream of its own."""
    H, Hkv, D, page, M = 8, 2, 128, 32, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rows = torch.empty(M, (H + 2 * Hkv) * D, dtype=torch.bfloat16, device=DEV)
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split((H * D, Hkv * D, Hkv * D), 1))
    numbers = [torch.zeros(M * 4, Hkv, page, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    scales = [torch.zeros(M * 4, Hkv, page // BLOCK, device=DEV) for _ in range(2)]
    cache = B.PagedCacheQ8(numbers[0], numbers[1], scales[0], scales[1])
    table = torch.randperm(M * 4, device=DEV).to(torch.int32).view(M, 4)
    positions = torch.zeros(M, dtype=torch.int32, device=DEV)
    batch = B.PagedBatch(positions, torch.arange(M + 1, dtype=torch.int32, device=DEV), table, M, 1)
    inv, status = torch.full((D // 2,), 0.01, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    turned, out = (torch.empty(M, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = B.paged_attention_q8_workspace(cache, batch, H)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        B.kvs_rope_scatter_paged_q8(q, k, v, turned, cache, batch, inv, d_status=status)
        B.kvs_paged_attention_q8(turned, cache, batch, out, workspace=ws, d_status=status)
        positions.add_(1)
    for t in range(40):
        rows.normal_(generator=g)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.current_stream().wait_stream(stream)
        if t in (0, 15, 16, 31, 32, 39):
            for i in range(M):
                kk, vv = ((x[table[i].long()].double() * s[table[i].long()].double().repeat_interleave(BLOCK, 2)[..., None])
                          .transpose(0, 1).reshape(Hkv, -1, D)[:, :t + 1] for x, s in zip(numbers, scales))
                z = torch.einsum("ged,gld->gel", turned[i].double().view(Hkv, H // Hkv, D), kk) / math.sqrt(D)
                ref = torch.einsum("gel,gld->ged", torch.softmax(z, -1), vv).reshape(H, D)
                # scores: sums of D products in steps of 16, three times 2^-23 an addition; two float16
                # parts of a weight and sums under 2^-16; a rounding to the type
                size = torch.einsum("ged,gld->gel", turned[i].double().abs().view(Hkv, H // Hkv, D), kk.abs()).amax()
                ds = size / math.sqrt(D) * (3 * D / 8 + 4) * 2.0 ** -23
                tol = (2 * ds + 2.0 ** -16) * vv.abs().amax() + 2.0 ** -8 * ref.abs() * 1.01
                within(out[i], ref, tol, f"step {t}, sequence {i}")
    assert int(status.item()) == 0 and int(positions[0].item()) == 40


def test_sampling_on_two_streams_and_threads():
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    xs = [torch.empty(9, 50001, dtype=t, device=DEV).normal_(generator=g) * 3 for t in (torch.float32, torch.bfloat16)]
    us = [torch.rand(9, device=DEV, generator=g) for _ in xs]
    p = torch.full((9,), 0.9, device=DEV)
    want = [B.kvs_sample_logits(x, u, top_p=p).clone() for x, u in zip(xs, us)]
    streams, outs, errors = [torch.cuda.Stream() for _ in xs], [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()

    def work(i):
        try:
            for _ in range(50):
                B.kvs_sample_logits(xs[i], us[i], token_ids=outs[i], top_p=p, stream=streams[i])
        except Exception as e:  # told to the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and all(torch.equal(a, b) for a, b in zip(want, outs))


def test_more_sampled_rows_than_a_grid_holds():
    """Rows past 65,535, the largest second dimension of a grid."""
    M, V = 70000, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    x = torch.empty(M, V, device=DEV).normal_(generator=g)
    ids = B.kvs_sample_logits(x, torch.zeros(M, device=DEV), top_k=torch.ones(M, dtype=torch.int32, device=DEV))
    assert torch.equal(ids.long(), x.argmax(1))
    u = torch.rand(M, device=DEV, generator=g)
    got = B.kvs_sample_logits(x, u).long()
    c = torch.softmax(x.double(), 1).cumsum(1)
    inside = c.gather(1, got[:, None])[:, 0] > u.double() - 1e-9
    before = torch.where(got > 0, c.gather(1, (got - 1).clamp_min(0)[:, None])[:, 0], torch.zeros_like(c[:, 0]))
    assert (inside & (before <= u.double() + 1e-9)).all()


def test_no_call_allocates():
    b, f = kind("chunks", seed=2), kind("long f32", seed=2)
    x, u, ids = torch.randn(5, 30000, device=DEV), torch.rand(5, device=DEV), torch.empty(5, dtype=torch.int32, device=DEV)
    outs = [torch.empty_like(b.q), torch.empty_like(f.q)]
    torch.cuda.synchronize()
    held = torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        b.attend(out=outs[0])
        f.attend(out=outs[1])
        B.kvs_sample_logits(x, u, token_ids=ids)
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == held
    b.check(outs[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [0.01, 4.0])
def test_sampling_from_the_largest_vocabulary(dtype, spread):
    """2^19 tokens, of nearly equal logits and of few that count, under each rule alone."""
    M, V = 3, 2 ** 19
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    x = (torch.empty(M, V, device=DEV).normal_(generator=g) * spread).to(DTYPES[dtype])
    u = torch.tensor([0.1, 0.5, 0.999], device=DEV)
    w = torch.softmax(x.double(), 1)
    order = torch.sort(x.double(), dim=1, descending=True, stable=True)[1]
    full = lambda v, t=torch.float32: torch.full((M,), v, dtype=t, device=DEV)
    for rules, count in ((dict(), V), (dict(top_k=full(700, torch.int32)), 700), (dict(top_p=full(0.5)), None)):
        ranked = w.gather(1, order)
        sums = ranked.cumsum(1)
        keep = torch.arange(V, device=DEV) < count if count else (sums - ranked) < 0.5 * sums[:, -1:]
        kept = torch.zeros_like(w).scatter_(1, order, ranked * keep)
        c = kept.cumsum(1) / kept.sum(1, keepdim=True)
        got = B.kvs_sample_logits(x, u, **rules).long()[:, None]
        low = c.gather(1, got) - kept.gather(1, got) / kept.sum(1, keepdim=True)
        # weights to 2^-37 of themselves; sums of 2^19 numbers of 64 bits here
        slack = 2.0 ** -30
        assert (low <= u[:, None].double() + slack).all() and (c.gather(1, got) >= u[:, None].double() - slack).all()
        assert (kept.gather(1, got) > 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [3000, 40001, 152064])
@pytest.mark.parametrize("spread", [0.001, 1.0, 30.0])
def test_sampling_from_the_first_few(dtype, V, spread):
    """Numbers of kept tokens around those that decide how they are found, for logits that hardly
    differ (and often tie), usual ones and steep ones."""
    ks = [2, 3, 20, 63, 64, 65, 128, 129, 255, 256, 257, 400]
    M = len(ks)
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    x = (torch.empty(M, V, device=DEV).normal_(generator=g) * spread).to(DTYPES[dtype])
    u = torch.rand(M, device=DEV, generator=g)
    k = torch.tensor(ks, dtype=torch.int32, device=DEV)
    prob = torch.empty(M, device=DEV)
    got = B.kvs_sample_logits(x, u, top_k=k, token_probs=prob).long()[:, None]
    order = torch.sort(x.double(), dim=1, descending=True, stable=True)[1]
    ranked = torch.softmax(x.double(), 1).gather(1, order) * (torch.arange(V, device=DEV) < k[:, None])
    w = torch.zeros(M, V, dtype=torch.float64, device=DEV).scatter_(1, order, ranked)
    w /= w.sum(1, keepdim=True)
    c = w.cumsum(1)
    p = w.gather(1, got)
    # weights to 2^-37 of themselves, those below 2^-45 of the largest as zero
    assert (p > 0).all()
    assert (c.gather(1, got) - p <= u[:, None].double() + 2.0 ** -30).all()
    assert (c.gather(1, got) >= u[:, None].double() - 2.0 ** -30).all()
    within(prob, p[:, 0], p[:, 0] * 2.0 ** -23 + 2.0 ** -44)
    probs = torch.empty(M, V, device=DEV)
    again = B.kvs_sample_logits(x, u, top_k=k, probs=probs).long()[:, None]
    assert torch.equal(got, again)
    within(probs, w, w * 2.0 ** -21 + 2.0 ** -44)
