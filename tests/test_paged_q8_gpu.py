"""kvs_paged_attention_q8 against the definition in 64 bits: types, head layouts, page sizes, chunk
and decode lengths, strides, scales far apart, bad input, graphs, streams."""
import math

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, within
from q8_helpers import BLOCK, E4M3, PagedQ8
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


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
                                          (8, 1, 128, 128), (3, 3, 64, 32), (6, 2, 128, 256),
                                          (5, 5, 128, 16)])
def test_matches_definition(batch, dtype, H, Hkv, D, page):
    n, p = BATCHES[batch]
    b = PagedQ8(n, p, H, Hkv, D, dtype, page, seed=len(batch) * 1000 + H * 10 + page)
    b.check(b.attend(), f"{batch} {dtype} {H}/{Hkv} {D} {page}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 257])
def test_every_tile_edge(dtype, n):
    """Chunk lengths and positions around the row and key tiles' borders."""
    for p in (0, n % 7, 127, 128):
        b = PagedQ8([n], [p], 8, 2, 64, dtype, 16, seed=n + p)
        b.check(b.attend(), f"{n} at {p}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("spread,powers", [(12, True), (2, False)])
def test_scales_far_apart_and_of_any_value(dtype, n, spread, powers):
    """Blocks whose scales differ by up to 2^24 (v's then decide the output beside the weights), and
    scales that are no powers of two."""
    b = PagedQ8([n, n], [333, 70], 8, 2, 128, dtype, 32, seed=spread + n, spread=spread, powers=powers)
    if spread > 2:  # scores of that size would leave one key only
        b.k_scales.copy_(torch.where(b.k_scales > 0, 2.0 ** -8, b.k_scales))
        b.q *= 0.25
        for i in range(2):
            L = n + b.p[i]
            pages = b.table_host[i, :-(-L // 32)]
            x = b.k_pages[pages.tolist()].double() * 2.0 ** -8
            b.k[i] = x.transpose(0, 1).reshape(2, -1, 128)[:, :L]
    b.check(b.attend(), f"{dtype} {n} {spread}")


@pytest.mark.parametrize("n", [1, 40])
def test_zero_rows_and_zero_scales(n):
    """A cache made of zeros, scales among them: every value is 0."""
    b = PagedQ8([n], [100], 8, 2, 64, "bf16", 16, seed=4)
    for t in (b.k_pages.view(torch.uint8), b.v_pages.view(torch.uint8), b.k_scales, b.v_scales):
        t.zero_()
    assert (b.attend() == 0).all()
    # zero rows of v beside others: the weights count, the rows do not
    b = PagedQ8([n], [100], 8, 2, 64, "bf16", 16, seed=5)
    first = int(b.table_host[0, 0])
    b.v_scales[first] = 0
    b.v[0][:, :16] = 0
    b.check(b.attend(), "first block of v without a scale")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_and_small_queries(dtype):
    """Rows of q near the ends of their type's range: their factor is a power of two."""
    for power in (-40, -12, 12) if dtype == "bf16" else (-12, 10):
        b = PagedQ8([1, 33], [50, 20], 4, 2, 64, dtype, 16, seed=8)
        b.k_scales.mul_(2.0 ** -power)
        b.q.mul_(2.0 ** power)
        b.k = [x * 2.0 ** -power for x in b.k]
        b.check(b.attend(), f"2^{power}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_chunk_over_long_context(dtype):
    b = PagedQ8([700, 1, 350], [3300, 8000, 0], 32, 8, 128, dtype, 64, seed=3)
    b.check(b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,p", [([1, 1, 1], [20011, 15000, 5003]), ([1], [40000]),
                                 ([1] * 9, list(range(100, 4600, 500)))])
def test_long_decodes_split_over_blocks(dtype, n, p):
    b = PagedQ8(n, p, 16, 4, 128, dtype, 64, seed=len(n))
    b.check(b.attend())
    again = b.attend()
    assert torch.equal(again, b.attend())


def test_strided_rows():
    b = PagedQ8([3, 1, 20], [40, 7, 300], 8, 2, 64, "bf16", 16, seed=9)
    wide = torch.full((b.rows, 3 * 8 * 64), 7.0, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 512:1024].unflatten(1, (8, 64))
    q.copy_(b.q)
    out = wide[:, 1024:].unflatten(1, (8, 64))
    b.attend(out=out, q=q)
    b.check(out, "strided")
    assert (wide[:, :512] == 7).all()


def test_rows_behind_the_last_sequence_stay():
    for n in ([1, 1], [30, 1]):
        b = PagedQ8(n, [5, 66], 8, 2, 64, "f16", 16, seed=2, tail_rows=4)
        out = b.attend()
        b.check(out)
        assert (out[sum(n):] == 7).all()


@pytest.mark.parametrize("n", [1, 33])
def test_bad_sequences_and_pages(n):
    """A bad position: NaN rows; a bad page: NaN rows that attend it; others as ever."""
    b = PagedQ8([n, n, n], [40, 100, 70], 8, 2, 64, "bf16", 16, seed=6)
    good, bound = b.reference()
    b.positions[1] = -1
    out = b.attend()
    assert int(b.status.item()) == B.KVS_ERR_POSITION
    assert torch.isnan(out[n:2 * n]).all()
    keep = torch.cat((torch.arange(n), torch.arange(2 * n, 3 * n))).to(DEV)
    within(out[keep], good[keep], bound[keep], "beside a bad position")
    b.positions[1] = 100
    b.status.zero_()
    b.page_table[1, 2] = 1 << 20
    out = b.attend()
    assert int(b.status.item()) == B.KVS_ERR_PAGE
    assert torch.isnan(out[n:2 * n]).all()
    within(out[keep], good[keep], bound[keep], "beside a bad page")
    b.status.zero_()
    b.row_offsets[1] = 3 * n + 1
    b.attend()
    assert int(b.status.item()) == B.KVS_ERR_ROWS


@pytest.mark.parametrize("n", [[1, 1, 1], [60, 1, 9]])
def test_captured_call_follows_its_inputs(n):
    b = PagedQ8(n, [900, 33, 0], 8, 2, 128, "bf16", 32, seed=12)
    out = b.attend()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        b.attend(out=out)
    out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    b.positions[0] = 500  # a shorter context of the same pages
    b.p[0] = 500
    b.k[0], b.v[0] = b.k[0][:, :500 + n[0]], b.v[0][:, :500 + n[0]]
    g.replay()
    torch.cuda.synchronize()
    b.check(out, "replayed on other positions")


def test_two_streams_with_workspaces_of_their_own():
    bs = [PagedQ8([1] * 4, [3000, 2000, 1000, 500], 8, 2, 128, "f16", 64, seed=s) for s in (1, 2)]
    want = [b.attend().clone() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    outs = [torch.zeros_like(w) for w in want]
    for _ in range(20):
        for b, s, o in zip(bs, streams, outs):
            b.attend(out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_more_sequences_than_blocks():
    rng = np.random.default_rng(0)
    p = rng.integers(0, 300, 500).tolist()
    b = PagedQ8([1] * 500, p, 4, 2, 64, "bf16", 16, seed=21)
    b.check(b.attend())
    n = rng.integers(0, 4, 300).tolist()
    b = PagedQ8(n, p[:300], 16, 2, 64, "bf16", 16, seed=22)
    b.check(b.attend())


def test_binding_refuses_wrong_tensors():
    b = PagedQ8([2], [3], 4, 2, 64, "f16", 16, seed=1)
    ok = dict(out=None, workspace=b.workspace)
    out = torch.empty_like(b.q)
    with pytest.raises(TypeError):
        B.kvs_paged_attention_q8(b.q.double(), b.cache, b.batch, out, workspace=ok["workspace"])
    with pytest.raises(TypeError):
        B.kvs_paged_attention_q8(b.q, b.cache, b.batch, out.float(), workspace=ok["workspace"])
    with pytest.raises(ValueError):
        B.kvs_paged_attention_q8(b.q, b.cache, b.batch, out)
    with pytest.raises(ValueError):
        B.kvs_paged_attention_q8(b.q, b.cache, b.batch, b.q, workspace=ok["workspace"])
    with pytest.raises(B.KvsError):
        B.kvs_paged_attention_q8(b.q, b.cache, b.batch, out, workspace=b.workspace[:256])
    with pytest.raises(TypeError):
        B.PagedCacheQ8(b.k_pages.view(torch.uint8), b.v_pages, b.k_scales, b.v_scales)
    with pytest.raises(TypeError):
        B.PagedCacheQ8(b.k_pages, b.v_pages, b.k_scales[:, :, :0], b.v_scales)
    with pytest.raises(ValueError):
        B.PagedCacheQ8(b.k_pages, b.v_pages[:1], b.k_scales, b.v_scales)
