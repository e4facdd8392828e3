"""The paged-cache and logit entry points where a program meets them unprepared: first calls
inside a capture, many sequences and rows, shared pages, workspaces in turn, two threads."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, Paged, half_step, least_step, within
from split_flash_decoding_kvcachescatter_gb300 import binding as B
from test_logits_gpu import Rules, check as check_logits, logits
from test_rope_gpu import check as check_rope, make_case, rotate64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from paged_helpers import Paged, DEV
from split_flash_decoding_kvcachescatter_gb300 import binding as B
kinds = [Paged([1, 1], [300, 5], 8, 2, 64, "f16", 16), Paged([1, 1], [300, 5], 8, 2, 64, "f32", 16, columns=2 ** 15),
         Paged([70, 1], [3, 90], 8, 2, 128, "bf16", 32), Paged([70, 1], [3, 90], 8, 2, 64, "f32", 32)]
x = torch.randn(3, 1000, device=DEV)
y, ids = torch.empty_like(x), torch.empty(3, dtype=torch.int32, device=DEV)
inv, _ = B.kvs_rope_frequencies(64)
r = kinds[0]
new = [torch.randn(2, 2, 64, device=DEV).half() for _ in range(2)]
outs = [torch.zeros_like(b.q) for b in kinds]
turned = torch.zeros_like(r.q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for b, out in zip(kinds, outs):
        b.attend(out=out)
    B.kvs_rope_scatter_paged(r.q, new[0], new[1], turned, r.cache, r.batch, inv, d_status=r.status)
    B.kvs_process_logits(x, y, token_ids=ids)
graph.replay()
torch.cuda.synchronize()
for b, out in zip(kinds, outs):
    b.check(out)
assert torch.equal(x, y) and torch.equal(ids.long(), x.argmax(1))
print("fine")
"""


def test_first_calls_of_a_process_inside_a_capture():
    code = FIRST_CALL.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def many(seed, M=150):
    rng = np.random.default_rng(seed)
    n = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 9, 40], M)]
    return n, [int(x) for x in rng.integers(0, 300, M)]


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_sequences(dtype):
    n, p = many(1)
    b = make_case(n, p, 8, 2, 64, dtype, 16, seed=2, tail_rows=5)
    b.check(b.attend())
    inv, scale = B.kvs_rope_frequencies(64)
    k0, v0 = b.k_pages.clone(), b.v_pages.clone()
    out = torch.zeros_like(b.q)
    B.kvs_rope_scatter_paged(b.q, b.new_k, b.new_v, out, b.cache, b.batch, inv.to(DEV), d_status=b.status)
    assert int(b.status.item()) == 0
    check_rope(b, out, inv.to(DEV), False, scale, k0, v0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,D", [(12, 2, 64), (8, 4, 128), (4, 1, 128), (512, 64, 64), (31, 31, 64)])
@pytest.mark.parametrize("n,p", [([1, 1, 0, 1], [70, 0, 3, 400]), ([30, 1, 0, 100], [70, 0, 3, 40])])
def test_other_head_layouts(dtype, H, Hkv, D, n, p):
    b = Paged(n, p, H, Hkv, D, dtype, 16, seed=H + D)
    b.check(b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("max_new", [17, 500, 2 ** 20])
def test_bound_on_new_tokens_above_all(dtype, max_new):
    """A program that always passes the largest chunk: decode steps then take the chunk kernels."""
    b = Paged([1, 1, 2, 0, 1], [700, 0, 31, 2, 4000], 8, 2, 64, dtype, 32, seed=3)
    b.batch = B.PagedBatch(b.positions, b.row_offsets, b.page_table, b.rows, max_new)
    b.workspace = B.paged_attention_workspace(b.cache, b.batch, 8)
    b.check(b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 1, 9]])
def test_sequences_share_the_pages_of_a_prefix(dtype, n):
    page, shared = 16, 5
    b = Paged(n, [90, 83, 100], 8, 2, 64, dtype, page, seed=4)
    for i in (1, 2):
        b.page_table[i, :shared] = b.page_table[0, :shared]
        for mine, first in ((b.k, b.k), (b.v, b.v)):
            mine[i][:, :shared * page] = first[0][:, :shared * page]
    b.check(b.attend())


def test_one_workspace_for_chunks_and_decode_steps_and_their_graphs():
    """A program's one workspace: calls of every kernel in turn, eager and replayed."""
    kinds = [Paged([90, 1, 300], [700, 3000, 0], 16, 4, 64, "f16", 32, seed=5),
             Paged([1, 1, 1], [7000, 3000, 40], 16, 4, 64, "f16", 32, seed=6, columns=2 ** 14),
             Paged([1] * 3, [700, 300, 40], 16, 4, 64, "f16", 32, seed=7),
             Paged([50, 1], [700, 300], 16, 4, 64, "f32", 32, seed=8)]
    ws = max((b.workspace for b in kinds), key=lambda t: t.numel())
    graphs, outs = [], []
    for b in kinds:
        b.workspace = ws
        outs.append(torch.zeros_like(b.q))
    for b, out in zip(kinds, outs):
        b.attend(out=out)
    torch.cuda.synchronize()
    for b, out in zip(kinds, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            b.attend(out=out)
    for order in ((0, 1, 2, 3), (3, 1, 0, 0, 2, 1, 3), (1, 1, 0)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
            kinds[order[0]].attend()
        torch.cuda.synchronize()
        for i in order:
            kinds[i].check(outs[i], f"order {order}, {i}")


def test_two_threads():
    cases = [Paged([1] * 6, [900 + i for i in range(6)], 16, 4, 64, "bf16", 32, seed=9),
             Paged([120, 1, 7], [700, 3000, 0], 16, 4, 64, "bf16", 32, seed=10)]
    outs, streams, errors = [torch.zeros_like(b.q) for b in cases], [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()

    def work(i):
        try:
            for _ in range(30):
                cases[i].attend(out=outs[i], stream=streams[i])
        except Exception as e:  # told to the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for b, out in zip(cases, outs):
        b.check(out)


def test_without_a_status_word():
    b = Paged([1, 20], [30, 0], 8, 2, 64, "f16", 16, seed=11)
    out = torch.full_like(b.q, 7.0)
    B.kvs_paged_attention(b.q, b.cache, b.batch, out, workspace=b.workspace)
    b.check(out)
    b.page_table[0, 0] = -1
    B.kvs_paged_attention(b.q, b.cache, b.batch, out, workspace=b.workspace)
    assert out[0].isnan().all() and not out[1:].isnan().any()


def test_attention_over_its_own_queries_is_refused():
    b = Paged([1, 20], [30, 0], 8, 2, 64, "f16", 16, seed=12)
    with pytest.raises(ValueError):
        b.attend(out=b.q)


@pytest.mark.parametrize("V", [9, 40])
def test_more_logit_rows_than_a_grid_holds(V):
    M = 66001
    x = logits(M, V, "f32", seed=V)
    r = Rules(M, V, history=6, bias=0, seed=V)
    out = torch.empty_like(x)
    ids = B.kvs_process_logits(x, out, **r.kwargs())
    check_logits(x, out, ids, r)


def test_partial_overlaps_are_refused_and_column_blocks_are_not():
    b = make_case([1, 20], [30, 0], 8, 2, 64, "f16", 16, seed=12)
    wide = torch.zeros(b.rows, 2 * 512, dtype=b.dtype, device=DEV)
    heads = lambda t: t.unflatten(1, (8, 64))
    q, out, across = (heads(wide[:, a:a + 512]) for a in (0, 512, 256))
    q.copy_(b.q)
    b.check(b.attend(q=q, out=out))
    inv, _ = B.kvs_rope_frequencies(64)
    for call in (lambda: b.attend(q=q, out=across),
                 lambda: B.kvs_rope_scatter_paged(q, b.new_k, b.new_v, across, b.cache, b.batch, inv),
                 lambda: B.kvs_process_logits(wide[:, :512], wide[:, 500:1012])):
        with pytest.raises(B.KvsError) as e:
            call()
        assert e.value.status == B.KVS_ERR_OVERLAP
    assert torch.equal(q, b.q)


def test_more_rotated_rows_than_32_bit_thread_numbers():
    """2^24 rows are 2^31 threads of the rotary kernel: every sequence's rows are found and written."""
    N, D, page = 2 ** 24 + 300, 64, 2 ** 15
    n = [N - 257, 0, 256, 1]
    p = [0, 5, 3, 2 ** 20]
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    qkv = torch.empty(N, 3 * D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    q, k, v = (qkv[:, j * D:(j + 1) * D].unflatten(1, (1, D)) for j in range(3))
    pages = -(-n[0] // page)
    kp = torch.zeros(pages + 2, 1, page, D, dtype=torch.bfloat16, device=DEV)
    cache = B.PagedCache(kp, torch.zeros_like(kp))
    table = torch.zeros(4, pages, dtype=torch.int32, device=DEV)
    table[0] = torch.arange(pages, dtype=torch.int32, device=DEV)
    table[2], table[3] = pages, pages + 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    batch = B.PagedBatch(i32(p), i32(np.concatenate([[0], np.cumsum(n)])), table, N, max(n))
    status = i32([0])
    inv, _ = B.kvs_rope_frequencies(D)
    out = torch.zeros(N, 1, D, dtype=torch.bfloat16, device=DEV)
    B.kvs_rope_scatter_paged(q, k, v, out, cache, batch, inv, d_status=status)
    assert int(status.item()) == 0
    assert torch.equal(cache.v_pages[:pages].view(-1, D)[:n[0]], v[:n[0], 0])
    assert torch.equal(cache.v_pages[pages, 0, 3:259], v[n[0]:N - 1, 0])
    assert torch.equal(cache.v_pages[pages + 1, 0, 2 ** 20 % page], v[N - 1, 0])
    rows = torch.tensor([0, 1, 2 ** 23, 2 ** 24 - 1, 2 ** 24, n[0] - 1, n[0], N - 2, N - 1], device=DEV)
    pos = torch.tensor([0, 1, 2 ** 23, 2 ** 24 - 1, 2 ** 24, n[0] - 1, 3, 258, 2 ** 20], device=DEV)
    ref, size = rotate64(q[rows], pos, inv, False, 1.0)
    within(out[rows], ref, size * 2.0 ** -21 + half_step(out.dtype) * ref.abs() * 1.01 + least_step(out.dtype))


@pytest.mark.parametrize("dtype,n", [("f16", 1), ("f32", 1), ("f16", 40), ("f32", 40)])
def test_most_sequences_of_a_batch_are_empty(dtype, n):
    """The largest number of sequences, all but the first and the last without a token."""
    M = 2 ** 20
    b = Paged([n, 1], [700, 90], 8, 2, 64, dtype, 16, seed=13)
    wide = torch.zeros(M, b.page_table.shape[1], dtype=torch.int32, device=DEV)
    wide[0], wide[-1] = b.page_table[0], b.page_table[1]
    positions = torch.zeros(M, dtype=torch.int32, device=DEV)
    positions[0], positions[-1] = 700, 90
    offsets = torch.full((M + 1,), n, dtype=torch.int32, device=DEV)
    offsets[0], offsets[-1] = 0, n + 1
    b.batch = B.PagedBatch(positions, offsets, wide, b.rows, n)
    b.check(b.attend())
