"""kvs_paged_attention against the definition in 64 bits: types, head layouts,
page sizes, chunk and decode lengths, strides, bad input, graphs, streams."""
import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, Paged, within
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


# (new tokens, first positions): decode steps, prompts, chunks, mixtures; lengths of zero and one;
# ends inside a page, on its border and one past it; single and many key tiles
BATCHES = {
    "one key": ([1], [0]),
    "decode": ([1, 1, 1, 1, 1], [0, 15, 16, 130, 1027]),
    "few new": ([2, 1, 0, 2], [30, 0, 5, 777]),
    "prompt": ([37], [0]),
    "chunk": ([130, 1], [200, 63]),
    "mixed": ([1, 300, 0, 1, 17, 64], [511, 0, 99, 2000, 31, 64]),
    "long decode": ([1], [9000]),
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 2, 64, 16), (14, 2, 64, 64), (40, 8, 128, 32),
                                          (8, 1, 128, 128), (3, 3, 64, 32), (6, 2, 128, 256)])
def test_matches_definition(batch, dtype, H, Hkv, D, page):
    n, p = BATCHES[batch]
    b = Paged(n, p, H, Hkv, D, dtype, page, seed=len(batch) * 1000 + H * 10 + page)
    b.check(b.attend(), f"{batch} {dtype} {H}/{Hkv} {D} {page}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 257])
def test_every_tile_edge(dtype, n):
    """Chunk lengths and positions around the row and key tiles' borders."""
    for p in (0, n % 7, 127, 128):
        b = Paged([n], [p], 8, 2, 64, dtype, 16, seed=n + p)
        b.check(b.attend(), f"{n} at {p}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_chunk_over_long_context(dtype):
    b = Paged([700, 1, 350], [3300, 8000, 0], 32, 8, 128, dtype, 64, seed=3)
    b.check(b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,p", [([1, 1, 1], [20011, 15000, 5003]), ([1], [40000]),
                                 ([1] * 40, [900 + 7 * i for i in range(40)]),
                                 ([2, 0, 1], [31000, 5, 12345])])
def test_decode_over_every_block(dtype, n, p):
    """Enough keys to give every block of the decode kernel a long range."""
    b = Paged(n, p, 16, 8, 64, dtype, 64, seed=sum(n) + len(p))
    first = b.attend()
    b.check(first)
    for _ in range(5):
        assert torch.equal(b.attend(), first)


# A decode step chooses its kernel by the page table's width: a table with room for 2^19 keys a
# sequence takes the one for long caches, also when the live keys are few.
WIDE = 2 ** 19


@pytest.mark.parametrize("batch", [b for b in BATCHES if max(BATCHES[b][0]) <= 2])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 2, 64, 16), (14, 2, 64, 64), (40, 8, 128, 32),
                                          (8, 1, 128, 128), (3, 3, 64, 32), (6, 2, 128, 256)])
def test_decode_with_room_for_long_sequences(batch, dtype, H, Hkv, D, page):
    n, p = BATCHES[batch]
    b = Paged(n, p, H, Hkv, D, dtype, page, seed=len(batch) * 1000 + H * 10 + page,
              columns=WIDE // page)
    b.check(b.attend(), f"{batch} {dtype} {H}/{Hkv} {D} {page}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,D,most", [(16, 8, 64, 250), (16, 8, 64, 1100), (32, 8, 128, 120),
                                          (8, 8, 128, 400), (14, 2, 64, 700)])
def test_decode_of_many_sequences(dtype, H, Hkv, D, most):
    """More (sequence, kv head) pairs than blocks run at once; some sequences are empty."""
    n = [0 if i % 11 == 5 else 2 if i % 7 == 3 else 1 for i in range(83)]
    p = [(i * 37) % (most - 2) for i in range(83)]
    b = Paged(n, p, H, Hkv, D, dtype, 16, seed=most + D)
    first = b.attend()
    b.check(first)
    for _ in range(3):
        assert torch.equal(b.attend(), first)


@pytest.mark.parametrize("columns", [2, WIDE // 32])
@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_bad_input_and_short_waits(dtype, columns):
    """Bad pages and positions poison their sequence alone, and waits that run out are told."""
    n, p = [1, 2, 1] * 9, [5000, 3000, 2000, 300, 200, 100, 0, 1, 40] * 3
    for what in ("page", "position"):
        b = Paged(n, p, 8, 2, 64, dtype, 32, seed=19, columns=columns)
        (b.page_table[4] if what == "page" else b.positions[4:5])[:1] = 2 ** 31 - 1
        out = b.attend()
        assert int(b.status.item()) == (B.KVS_ERR_PAGE if what == "page" else B.KVS_ERR_POSITION)
        ref, bound = b.reference()
        a, e = int(b.offsets_host[4]), int(b.offsets_host[5])
        assert out[a:e].isnan().all()
        keep = [r for r in range(sum(n)) if not a <= r < e]
        within(out[keep], ref[keep], bound[keep], what)
    b = Paged(n, p, 8, 2, 64, dtype, 32, seed=20, columns=columns)
    prev = B.kvs_set_wait_limit_ns(0)
    try:
        b.attend()
        torch.cuda.synchronize()
        assert int(b.status.item()) == B.KVS_ERR_TIMEOUT
    finally:
        B.kvs_set_wait_limit_ns(prev)
    b.status.zero_()
    b.check(b.attend())


def test_wide_decode_graph_and_two_streams():
    """The kernel for long caches: replays of a capture, and two streams at once."""
    a = Paged([1] * 8, [4000 + 3 * i for i in range(8)], 32, 8, 128, "f16", 64, seed=21,
              columns=WIDE // 64)
    b = Paged([1, 2, 1], [9000, 10, 700], 16, 4, 64, "f32", 32, seed=22, columns=WIDE // 32)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(a.q), torch.empty_like(b.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.attend(out=oa)
    for _ in range(5):
        with torch.cuda.stream(s):
            graph.replay()
        b.attend(out=ob, stream=t)
    torch.cuda.synchronize()
    a.check(oa)
    b.check(ob)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_scores(dtype):
    """Scores of some hundreds: the running maximum moves often and far."""
    b = Paged([1, 90], [600, 500], 8, 2, 128, dtype, 32, seed=4)
    # ascending keys, so that the maximum moves in almost every tile
    for i in range(2):
        L = b.k[i].shape[1]
        ramp = torch.linspace(0.1, 8.0, L, device=DEV)[:, None].to(b.dtype)
        b.k[i].mul_(ramp)
        for j in range(-(-L // 32)):
            a, e = j * 32, min(L, (j + 1) * 32)
            b.k_pages[b.table_host[i, j], :, :e - a] = b.k[i][:, a:e]
    b.check(b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,p", [([1, 1], [40, 300]), ([70, 3], [5, 200])])
def test_strided_rows_and_rows_behind_the_last_sequence(dtype, n, p):
    b = Paged(n, p, 8, 2, 64, dtype, 16, seed=5, tail_rows=3)
    wide = torch.full((b.rows, 8 * 64 + 24), 3.0, dtype=b.dtype, device=DEV)
    wide[:, 8:8 + 512] = b.q.view(b.rows, 512)
    q = wide[:, 8:8 + 512].unflatten(1, (8, 64))
    out_wide = torch.full((b.rows, 8 * 64 + 8), 7.0, dtype=b.dtype, device=DEV)
    out = out_wide[:, :512].unflatten(1, (8, 64))
    b.attend(out=out, q=q)
    b.check(out)
    assert (out_wide[:, 512:] == 7).all(), "wrote between the rows"
    assert (out_wide[sum(n):] == 7).all(), "wrote behind the last sequence"


def test_pages_past_32_bit_offsets():
    """The live pages lie past 2^32 bytes and 2^31 elements of the pool."""
    Hkv, page, D = 8, 256, 128
    pages = 9000  # 512 KB each in float16
    b = Paged([1, 40], [700, 300], 16, Hkv, D, "f16", page, seed=6)
    k = torch.empty(pages, Hkv, page, D, dtype=b.dtype, device=DEV)
    v = torch.empty_like(k)
    used = b.k_pages.shape[0]
    k[-used:], v[-used:] = b.k_pages, b.v_pages
    table = torch.where(b.page_table >= 0, b.page_table + (pages - used), b.page_table)
    b.page_table.copy_(table)
    b.cache = B.PagedCache(k, v)
    b.check(b.attend())


@pytest.mark.parametrize("n", [[1, 1, 1], [70, 1, 40]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_page(dtype, n):
    for bad in (-1, 10 ** 6):
        b = Paged(n, [300, 200, 100], 8, 2, 64, dtype, 32, seed=7)
        b.page_table[1, 2] = bad
        out = b.attend()
        assert int(b.status.item()) == B.KVS_ERR_PAGE
        ref, bound = b.reference()
        a, e = n[0], n[0] + n[1]
        assert out[a:e].isnan().all()
        keep = [r for r in range(sum(n)) if not a <= r < e]
        within(out[keep], ref[keep], bound[keep])


@pytest.mark.parametrize("n", [[1, 1, 1], [70, 1, 40]])
def test_bad_position(n):
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        b = Paged(n, [300, 200, 100], 8, 2, 64, "f16", 32, seed=8)
        b.positions[1] = bad
        out = b.attend()
        assert int(b.status.item()) == B.KVS_ERR_POSITION
        ref, bound = b.reference()
        a, e = n[0], n[0] + n[1]
        assert out[a:e].isnan().all()
        keep = [r for r in range(sum(n)) if not a <= r < e]
        within(out[keep], ref[keep], bound[keep])


def test_bad_row_offsets():
    n = [3, 2, 4]
    for at, value in ((1, -1), (2, 1), (3, 1000), (0, -5)):
        b = Paged(n, [30, 20, 10], 8, 2, 64, "f32", 32, seed=9)
        b.row_offsets[at] = value
        out = b.attend()
        assert int(b.status.item()) == B.KVS_ERR_ROWS
        assert not out.isnan().any()
    b = Paged(n, [30, 20, 10], 8, 2, 64, "f32", 32, seed=9)
    small = B.PagedBatch(b.positions, b.row_offsets, b.page_table, b.rows, 3)  # sequence 2 has 4
    out = torch.full_like(b.q, 7.0)
    B.kvs_paged_attention(b.q, b.cache, small, out, workspace=b.workspace, d_status=b.status)
    assert int(b.status.item()) == B.KVS_ERR_ROWS
    assert (out[5:] == 7).all()
    ref, bound = b.reference()
    within(out[:5], ref[:5], bound[:5])


def test_empty_calls():
    b = Paged([0, 0], [3, 4], 8, 2, 64, "f32", 32, seed=10, tail_rows=2)
    assert (b.attend() == 7).all() and int(b.status.item()) == 0
    q = torch.empty(0, 8, 64, device=DEV)
    batch = B.PagedBatch(b.positions, b.row_offsets, b.page_table, 0, 1)
    B.kvs_paged_attention(q, b.cache, batch, q, workspace=b.workspace)


@pytest.mark.parametrize("dtype", DTYPES)
def test_same_bits_every_time(dtype):
    b = Paged([1, 200, 1, 1], [5000, 100, 3000, 17], 32, 8, 128, dtype, 64, seed=11)
    first = b.attend()
    b.workspace.random_(0, 255)  # whatever the workspace held
    for _ in range(3):
        assert torch.equal(b.attend(), first)


@pytest.mark.parametrize("n,p,q", [([1, 1, 1], [100, 900, 40], [2000, 3, 777]),
                                   ([50, 1, 100], [100, 900, 40], [50, 1200, 0]),
                                   ([1, 1, 1], [50000, 9000, 31000], [20, 70000, 20000])])
def test_graph_follows_positions(n, p, q):
    """A captured call replays on other positions, with a batch's tables rewritten in place."""
    big = [max(a, c) for a, c in zip(p, q)]
    shape = Paged(n, big, 16, 4, 64, "bf16", 32, seed=12)
    batches = [Paged(n, x, 16, 4, 64, "bf16", 32, seed=s, spare=80) for s, x in ((13, p), (14, q))]
    size = max(b.k_pages.shape[0] for b in batches)
    k = torch.zeros(size, 4, 32, 64, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    out = torch.empty_like(shape.q)
    qin = torch.empty_like(shape.q)
    shape.cache = B.PagedCache(k, v)

    def load(b):
        k[:b.k_pages.shape[0]], v[:b.k_pages.shape[0]] = b.k_pages, b.v_pages
        shape.page_table.fill_(-1)
        w = min(shape.page_table.shape[1], b.page_table.shape[1])
        shape.page_table[:, :w] = b.page_table[:, :w]
        shape.positions.copy_(b.positions)
        qin.copy_(b.q)

    load(batches[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        shape.attend(out=out, q=qin)  # set-up before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        shape.attend(out=out, q=qin)
    for b in batches + batches[:1]:
        load(b)
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(shape.status.item()) == 0
        b.check(out)


def test_two_streams_with_workspaces_of_their_own():
    a = Paged([1] * 8, [4000 + 3 * i for i in range(8)], 32, 8, 128, "f16", 64, seed=15)
    b = Paged([120, 1], [700, 9], 32, 8, 128, "f16", 64, seed=16)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(a.q), torch.empty_like(b.q)
    for _ in range(5):
        a.attend(out=oa, stream=s)
        b.attend(out=ob, stream=t)
    torch.cuda.synchronize()
    a.check(oa)
    b.check(ob)


@pytest.mark.parametrize("n", [[1] * 4, [200, 3, 1, 1]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_waits_that_run_out_are_reported(dtype, n):
    """With the wait bound at zero some wait of some block runs out: the status says so, and
    the same workspace serves the next call."""
    b = Paged(n, [5000, 3000, 2000, 700], 16, 4, 128, dtype, 32, seed=17)
    prev = B.kvs_set_wait_limit_ns(0)
    try:
        b.attend()
        torch.cuda.synchronize()
        assert int(b.status.item()) == B.KVS_ERR_TIMEOUT
    finally:
        B.kvs_set_wait_limit_ns(prev)
    b.status.zero_()
    b.check(b.attend())


def test_refusals_of_the_binding():
    b = Paged([2], [3], 4, 2, 64, "f32", 16, seed=18)
    out = torch.empty_like(b.q)
    ok = dict(workspace=b.workspace)
    with pytest.raises(ValueError):
        B.kvs_paged_attention(b.q, b.cache, b.batch, out)
    with pytest.raises(TypeError):
        B.kvs_paged_attention(b.q.half(), b.cache, b.batch, out, **ok)
    with pytest.raises(TypeError):
        B.kvs_paged_attention(b.q[:1], b.cache, b.batch, out, **ok)
    with pytest.raises(TypeError):
        B.kvs_paged_attention(b.q.transpose(1, 2).contiguous().transpose(1, 2), b.cache, b.batch,
                              out, **ok)
    with pytest.raises(B.KvsError) as e:
        B.kvs_paged_attention(b.q, b.cache, b.batch, out, workspace=b.workspace[:256])
    assert e.value.status == B.KVS_ERR_WORKSPACE
    with pytest.raises(TypeError):
        B.PagedCache(b.k_pages.double(), b.v_pages.double())
    with pytest.raises(ValueError):
        B.PagedCache(b.k_pages, b.v_pages[:1])
    with pytest.raises(ValueError):
        B.PagedBatch(b.positions, b.row_offsets[:1], b.page_table, 2, 2)
