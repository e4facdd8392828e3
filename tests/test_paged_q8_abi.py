"""Host-side checks of the 8-bit paged cache's entry points and of the choice of
a token that need no GPU: refusals before CUDA is touched, workspace sizes."""
import ctypes

import pytest
import torch

from split_flash_decoding_kvcachescatter_gb300 import binding as B
from split_flash_decoding_kvcachescatter_gb300 import build as kbuild

A16 = 1 << 20  # an aligned fake address; never dereferenced (validation fails first)
BIG = 1 << 40  # another, far from it


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return B.lib()


def cache(k=A16, v=A16, ks=A16, vs=A16, pages=4, page=16, Hkv=2, D=64):
    return B._PagedCacheQ8Struct(k, v, ks, vs, pages, page, Hkv, D)


def batch(pos=A16, off=A16, table=A16, M=2, rows=5, max_new=3, max_pages=4):
    return B._PagedBatchStruct(pos, off, table, M, rows, max_new, max_pages)


def addr(s):
    return ctypes.addressof(s) if s is not None else None


def attend(L, c, b, q=A16, qs=256, dtype=B.KVS_BF16, out=BIG, os_=256, H=4, ws=A16, wsb=1 << 30):
    return L.kvs_paged_attention_q8(q, qs, dtype, addr(c), addr(b), out, os_, H, ws, wsb, None, None)


def rope(L, c, b, q=A16, qs=256, k=A16, ks=128, v=A16, vs=128, o=BIG, os_=256, dtype=B.KVS_BF16,
         inv=A16, H=4, rot=64):
    return L.kvs_rope_scatter_paged_q8(q, qs, k, ks, v, vs, o, os_, dtype, addr(c), addr(b), inv, H,
                                       rot, 0, 1.0, None, None)


@pytest.mark.parametrize("ckw,bkw,kw,code", [
    (dict(pages=0), {}, {}, B.KVS_ERR_DIMS), (dict(page=0), {}, {}, B.KVS_ERR_DIMS),
    (dict(Hkv=0), {}, {}, B.KVS_ERR_DIMS), (dict(Hkv=3), {}, {}, B.KVS_ERR_DIMS),
    (dict(pages=1 << 28), {}, {}, B.KVS_ERR_DIMS),
    (dict(page=8), {}, {}, B.KVS_ERR_UNSUPPORTED), (dict(page=48), {}, {}, B.KVS_ERR_UNSUPPORTED),
    (dict(D=96), {}, {}, B.KVS_ERR_UNSUPPORTED),
    ({}, {}, dict(dtype=3), B.KVS_ERR_UNSUPPORTED), ({}, {}, dict(dtype=-1), B.KVS_ERR_UNSUPPORTED),
    ({}, {}, dict(H=18), B.KVS_ERR_UNSUPPORTED), ({}, {}, dict(H=0), B.KVS_ERR_DIMS),
    ({}, dict(M=-1), {}, B.KVS_ERR_DIMS), ({}, dict(rows=-1), {}, B.KVS_ERR_DIMS),
    ({}, dict(max_new=0), {}, B.KVS_ERR_DIMS), ({}, dict(max_pages=0), {}, B.KVS_ERR_DIMS),
    ({}, dict(max_pages=1 << 27), {}, B.KVS_ERR_DIMS),
    ({}, dict(M=(1 << 20) + 1, rows=0), {}, B.KVS_ERR_UNSUPPORTED),
    (dict(k=None), {}, {}, B.KVS_ERR_NULL), (dict(v=None), {}, {}, B.KVS_ERR_NULL),
    (dict(ks=None), {}, {}, B.KVS_ERR_NULL), (dict(vs=None), {}, {}, B.KVS_ERR_NULL),
    ({}, dict(pos=None), {}, B.KVS_ERR_NULL), ({}, dict(off=None), {}, B.KVS_ERR_NULL),
    ({}, dict(table=None), {}, B.KVS_ERR_NULL), ({}, {}, dict(q=None), B.KVS_ERR_NULL),
    (dict(k=A16 + 8), {}, {}, B.KVS_ERR_ALIGN), (dict(v=A16 + 8), {}, {}, B.KVS_ERR_ALIGN),
    (dict(ks=A16 + 2), {}, {}, B.KVS_ERR_ALIGN), (dict(vs=A16 + 1), {}, {}, B.KVS_ERR_ALIGN),
    ({}, dict(table=A16 + 2), {}, B.KVS_ERR_ALIGN), ({}, {}, dict(q=A16 + 8), B.KVS_ERR_ALIGN),
    ({}, {}, dict(qs=260), B.KVS_ERR_ALIGN), ({}, {}, dict(qs=255), B.KVS_ERR_DIMS),
    ({}, {}, dict(os_=255), B.KVS_ERR_DIMS), ({}, {}, dict(os_=260), B.KVS_ERR_ALIGN),
    ({}, dict(M=0), {}, B.KVS_OK), ({}, dict(rows=0), {}, B.KVS_OK),
    (dict(ks=None, k=None), dict(rows=0), {}, B.KVS_OK), ({}, dict(M=1 << 20, rows=0), {}, B.KVS_OK),
])
def test_both_check_the_cache_the_batch_and_the_rows(L, ckw, bkw, kw, code):
    assert attend(L, cache(**ckw), batch(**bkw), **kw) == code
    assert rope(L, cache(**ckw), batch(**bkw), **kw) == code


def test_null_structs(L):
    for c, b in ((None, batch()), (cache(), None)):
        assert attend(L, c, b) == B.KVS_ERR_NULL
        assert rope(L, c, b) == B.KVS_ERR_NULL


@pytest.mark.parametrize("kw,code", [
    (dict(out=None), B.KVS_ERR_NULL), (dict(out=BIG + 8), B.KVS_ERR_ALIGN),
    (dict(ws=None), B.KVS_ERR_WORKSPACE), (dict(ws=A16 + 128), B.KVS_ERR_ALIGN),
    (dict(wsb=0), B.KVS_ERR_WORKSPACE), (dict(wsb=1000), B.KVS_ERR_WORKSPACE),
    # rows of 512 bytes, in the 16-bit types: the last byte of a row, one row on, the row's end
    (dict(out=A16), B.KVS_ERR_OVERLAP), (dict(out=A16 + 496), B.KVS_ERR_OVERLAP),
    (dict(out=A16 + 4 * 512), B.KVS_ERR_OVERLAP), (dict(out=A16 - 4 * 512 - 496), B.KVS_ERR_OVERLAP),
    (dict(qs=512, os_=512, out=A16 + 256), B.KVS_ERR_OVERLAP),
])
def test_attention_refusals(L, kw, code):
    assert attend(L, cache(), batch(), **kw) == code


@pytest.mark.parametrize("page", [16, 4096, 1 << 20])
def test_attention_keeps_clear_of_32_bit_key_counts(L, page):
    most = (2 ** 31 - 4096) // page
    if (most + 1) * page < 2 ** 31:
        above = batch(rows=0, max_pages=most + 1)
        assert attend(L, cache(pages=1, page=page), above) == B.KVS_ERR_DIMS
        assert rope(L, cache(pages=1, page=page), above) == B.KVS_OK
    assert attend(L, cache(pages=1, page=page), batch(rows=0, max_pages=most)) == B.KVS_OK


@pytest.mark.parametrize("kw,code", [
    (dict(rot=-2), B.KVS_ERR_DIMS), (dict(rot=63), B.KVS_ERR_DIMS), (dict(rot=66), B.KVS_ERR_DIMS),
    (dict(k=None), B.KVS_ERR_NULL), (dict(v=None), B.KVS_ERR_NULL), (dict(o=None), B.KVS_ERR_NULL),
    (dict(inv=None), B.KVS_ERR_NULL), (dict(inv=A16 + 1), B.KVS_ERR_ALIGN),
    (dict(ks=127), B.KVS_ERR_DIMS), (dict(vs=132), B.KVS_ERR_ALIGN), (dict(o=BIG + 8), B.KVS_ERR_ALIGN),
    (dict(o=A16 + 16), B.KVS_ERR_OVERLAP),                       # queries, not in place
    (dict(q=BIG, o=A16 + 4 * 256, k=A16), B.KVS_ERR_OVERLAP),    # the last row of k
    (dict(q=BIG, o=A16 - 4 * 512 - 496, k=2 * BIG), B.KVS_ERR_OVERLAP),  # the first row of v
])
def test_rope_refusals(L, kw, code):
    assert rope(L, cache(), batch(), **kw) == code


def test_workspace_bytes(L):
    f = L.kvs_paged_attention_q8_workspace_bytes
    assert f(4, 0, 64, 1) == 0 and f(5, 2, 64, 1) == 0 and f(4, 2, 96, 1) == 0
    assert f(4, 2, 64, 0) == 0 and f(18, 2, 64, 1) == 0 and f(-4, 2, 64, 1) == 0
    for H, Hkv, D in ((4, 2, 64), (40, 8, 128)):
        sizes = [f(H, Hkv, D, n) for n in (1, 2, 3, 4, 8, 16, 17, 1000, 2 ** 31 - 1)]
        assert all(0 < n < 64 << 20 for n in sizes)
        assert sizes == sorted(sizes)  # a workspace for longer chunks serves shorter ones
        assert sizes[-1] == sizes[-2]
        for n, m in ((1, sizes[0]), (1000, sizes[-2])):
            b = batch(max_new=n)
            c = cache(Hkv=Hkv, D=D)
            assert attend(L, c, b, qs=H * D, os_=H * D, H=H, wsb=m - 1) == B.KVS_ERR_WORKSPACE


def sample(L, x=A16, xs=1000, dtype=B.KVS_F32, M=2, V=1000, u=A16, ids=A16, tp=None, p=None, ps=1000,
           rules=True, **kw):
    r = ctypes.create_string_buffer(
        B._pack_sample(*(kw.get(n, 0) for n in ("temperature", "top_k", "top_p", "min_p"))))
    return L.kvs_sample_logits(x, xs, dtype, M, V, u, r if rules else None, ids, tp, p, ps, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=(1 << 30) + 1, x=None), B.KVS_ERR_UNSUPPORTED), (dict(M=1 << 30, x=None), B.KVS_ERR_NULL),
    (dict(M=-1), B.KVS_ERR_DIMS), (dict(V=0), B.KVS_ERR_DIMS), (dict(V=(1 << 19) + 1), B.KVS_ERR_UNSUPPORTED),
    (dict(dtype=7), B.KVS_ERR_UNSUPPORTED), (dict(x=None), B.KVS_ERR_NULL), (dict(u=None), B.KVS_ERR_NULL),
    (dict(ids=None), B.KVS_ERR_NULL), (dict(xs=999), B.KVS_ERR_DIMS), (dict(xs=-1000), B.KVS_ERR_DIMS),
    (dict(p=BIG, ps=999), B.KVS_ERR_DIMS), (dict(x=A16 + 2), B.KVS_ERR_ALIGN),
    (dict(x=A16 + 1, dtype=B.KVS_BF16), B.KVS_ERR_ALIGN), (dict(u=A16 + 2), B.KVS_ERR_ALIGN),
    (dict(ids=A16 + 2), B.KVS_ERR_ALIGN), (dict(tp=A16 + 2), B.KVS_ERR_ALIGN), (dict(p=BIG + 2), B.KVS_ERR_ALIGN),
    (dict(temperature=A16 + 2), B.KVS_ERR_ALIGN), (dict(top_k=A16 + 2), B.KVS_ERR_ALIGN),
    (dict(top_p=A16 + 2), B.KVS_ERR_ALIGN), (dict(min_p=A16 + 2), B.KVS_ERR_ALIGN),
    (dict(rules=False, ids=A16 + 2), B.KVS_ERR_ALIGN),
    (dict(p=A16), B.KVS_ERR_OVERLAP), (dict(p=A16 + 7996), B.KVS_ERR_OVERLAP),
    (dict(p=A16 - 7996), B.KVS_ERR_OVERLAP), (dict(p=A16 + 1996, dtype=B.KVS_F16), B.KVS_ERR_OVERLAP),
    (dict(M=0, x=None, u=None, ids=None), B.KVS_OK),
])
def test_sample_refusals(L, kw, code):
    assert sample(L, **kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch at made-up addresses")
@pytest.mark.parametrize("kw", [
    dict(p=A16 + 8000), dict(p=A16 - 8000), dict(p=A16 + 4000, dtype=B.KVS_F16),
    dict(p=A16 + 4000, xs=2000, ps=2000), dict(ids=None, tp=A16), dict(ids=None, p=BIG),
    dict(rules=False), dict(xs=1 << 40),
])
def test_sample_takes_what_lies_beside_the_logits(L, kw):
    """(There is no device to run on: what passes the checks ends there.)"""
    assert sample(L, **kw) == B.KVS_ERR_LAUNCH


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch at made-up addresses")
def test_rows_beside_each_other_pass(L):
    wide = dict(qs=512, os_=512)
    assert attend(L, cache(), batch(), out=A16 + 5 * 512) == B.KVS_ERR_LAUNCH
    assert attend(L, cache(), batch(), out=A16 + 512, **wide) == B.KVS_ERR_LAUNCH
    assert rope(L, cache(), batch(), q=BIG, k=A16 + 4096, v=A16 + 8192) == B.KVS_ERR_LAUNCH  # in place
    assert rope(L, cache(), batch(), q=BIG, o=A16 + 5 * 256) == B.KVS_ERR_LAUNCH


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_the_binding_refuses_host_tensors():
    pages, scales = torch.zeros(2, 1, 16, 64, dtype=torch.float8_e4m3fn), torch.ones(2, 1, 1)
    with pytest.raises(TypeError, match="k_pages"):
        B.PagedCacheQ8(pages, pages.clone(), scales, scales.clone())
    with pytest.raises(TypeError, match="logits"):
        B.kvs_sample_logits(torch.zeros(2, 8), torch.zeros(2))
