"""Host-side checks of the paged-cache and logit entry points that need no
GPU: refusals before CUDA is touched, workspace sizes, frequency tables."""
import ctypes

import numpy as np
import pytest
import torch

from split_flash_decoding_kvcachescatter_gb300 import binding as B
from split_flash_decoding_kvcachescatter_gb300 import build as kbuild

A16 = 1 << 20  # an aligned fake address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return B.lib()


def cache(k=A16, v=A16, pages=4, page=16, Hkv=2, D=64, dtype=B.KVS_F32):
    return B._PagedCacheStruct(k, v, pages, page, Hkv, D, dtype)


def batch(pos=A16, off=A16, table=A16, M=2, rows=5, max_new=3, max_pages=4):
    return B._PagedBatchStruct(pos, off, table, M, rows, max_new, max_pages)


SHAPES = [
    (dict(pages=0), {}, B.KVS_ERR_DIMS), (dict(page=0), {}, B.KVS_ERR_DIMS),
    (dict(Hkv=0), {}, B.KVS_ERR_DIMS), (dict(Hkv=3), {}, B.KVS_ERR_DIMS),
    (dict(page=8), {}, B.KVS_ERR_UNSUPPORTED), (dict(page=48), {}, B.KVS_ERR_UNSUPPORTED),
    (dict(D=96), {}, B.KVS_ERR_UNSUPPORTED), (dict(dtype=3), {}, B.KVS_ERR_UNSUPPORTED),
    (dict(dtype=-1), {}, B.KVS_ERR_UNSUPPORTED),
    (dict(pages=1 << 28), {}, B.KVS_ERR_DIMS),
    ({}, dict(M=-1), B.KVS_ERR_DIMS), ({}, dict(rows=-1), B.KVS_ERR_DIMS),
    ({}, dict(max_new=0), B.KVS_ERR_DIMS), ({}, dict(max_pages=0), B.KVS_ERR_DIMS),
    ({}, dict(max_pages=1 << 27), B.KVS_ERR_DIMS),
    (dict(k=None), {}, B.KVS_ERR_NULL), (dict(v=None), {}, B.KVS_ERR_NULL),
    ({}, dict(pos=None), B.KVS_ERR_NULL), ({}, dict(off=None), B.KVS_ERR_NULL),
    ({}, dict(table=None), B.KVS_ERR_NULL),
    (dict(k=A16 + 8), {}, B.KVS_ERR_ALIGN), ({}, dict(table=A16 + 2), B.KVS_ERR_ALIGN),
    ({}, dict(M=0), B.KVS_OK), ({}, dict(rows=0), B.KVS_OK),
    ({}, dict(M=(1 << 20) + 1, rows=0), B.KVS_ERR_UNSUPPORTED), ({}, dict(M=2 ** 31 - 1, rows=0), B.KVS_ERR_UNSUPPORTED),
    ({}, dict(M=1 << 20, rows=0), B.KVS_OK),
]


def addr(s):
    return ctypes.addressof(s) if s is not None else None


def attend(L, c, b, q=A16, qs=256, out=A16, os_=256, H=4, ws=A16, wsb=1 << 30):
    return L.kvs_paged_attention(q, qs, addr(c), addr(b), out, os_, H, ws, wsb, None, None)


def rope(L, c, b, q=A16, qs=256, k=A16, ks=128, v=A16, vs=128, o=A16, os_=256, inv=A16, H=4, rot=64,
         il=0):
    return L.kvs_rope_scatter_paged(q, qs, k, ks, v, vs, o, os_, addr(c), addr(b), inv, H, rot, il,
                                    1.0, None, None)


@pytest.mark.parametrize("ckw,bkw,code", SHAPES)
def test_cache_and_batch_validation(L, ckw, bkw, code):
    assert attend(L, cache(**ckw), batch(**bkw)) == code
    assert rope(L, cache(**ckw), batch(**bkw)) == code


@pytest.mark.parametrize("page", [16, 256, 4096, 1 << 20])
def test_attention_keeps_clear_of_32_bit_key_counts(L, page):
    """Lengths near 2^31 are reachable (a table may name one page many times), and the kernels look
    ahead of a key: the table's reach stays 4,096 below.  The scatter has no such need."""
    most = (2 ** 31 - 4096) // page
    for M in (0, 2):
        above = batch(M=M, rows=0, max_pages=most + 1)
        if (most + 1) * page < 2 ** 31:
            assert attend(L, cache(pages=1, page=page), above) == B.KVS_ERR_DIMS
            assert rope(L, cache(pages=1, page=page), above) == B.KVS_OK
        assert attend(L, cache(pages=1, page=page), batch(M=M, rows=0, max_pages=most)) == B.KVS_OK


def test_null_structs(L):
    assert attend(L, None, batch()) == B.KVS_ERR_NULL
    assert attend(L, cache(), None) == B.KVS_ERR_NULL
    assert rope(L, None, batch()) == B.KVS_ERR_NULL


@pytest.mark.parametrize("kw,code", [
    (dict(H=0), B.KVS_ERR_DIMS), (dict(H=5), B.KVS_ERR_DIMS), (dict(H=18, qs=4096, os_=4096), B.KVS_ERR_UNSUPPORTED),
    (dict(q=None), B.KVS_ERR_NULL), (dict(out=None), B.KVS_ERR_NULL),
    (dict(qs=255), B.KVS_ERR_DIMS), (dict(qs=257), B.KVS_ERR_ALIGN), (dict(os_=258), B.KVS_ERR_ALIGN),
    (dict(q=A16 + 4), B.KVS_ERR_ALIGN), (dict(ws=None), B.KVS_ERR_WORKSPACE),
    (dict(ws=A16 + 16), B.KVS_ERR_ALIGN), (dict(wsb=1000), B.KVS_ERR_WORKSPACE),
])
def test_paged_attention_validation(L, kw, code):
    assert attend(L, cache(), batch(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rot=-2), B.KVS_ERR_DIMS), (dict(rot=63), B.KVS_ERR_DIMS), (dict(rot=66), B.KVS_ERR_DIMS),
    (dict(q=None), B.KVS_ERR_NULL), (dict(k=None), B.KVS_ERR_NULL), (dict(v=None), B.KVS_ERR_NULL),
    (dict(o=None), B.KVS_ERR_NULL), (dict(inv=None), B.KVS_ERR_NULL), (dict(inv=A16 + 1), B.KVS_ERR_ALIGN),
    (dict(ks=127), B.KVS_ERR_DIMS), (dict(vs=130), B.KVS_ERR_ALIGN), (dict(o=A16 + 8), B.KVS_ERR_ALIGN),
])
def test_rope_validation(L, kw, code):
    assert rope(L, cache(), batch(), **kw) == code


def test_workspace_bytes(L):
    f = L.kvs_paged_attention_workspace_bytes
    assert f(4, 0, 64, 1) == 0 and f(5, 2, 64, 1) == 0 and f(4, 2, 96, 1) == 0
    assert f(4, 2, 64, 0) == 0 and f(18, 2, 64, 1) == 0
    for H, Hkv, D in ((4, 2, 64), (40, 8, 128)):
        small, large = f(H, Hkv, D, 1), f(H, Hkv, D, 1000)
        assert 0 < small < large < 64 << 20
        assert f(H, Hkv, D, 2 ** 31 - 1) == large


def logits(L, x=A16, xs=1000, o=A16, os_=1000, dtype=B.KVS_F32, M=2, V=1000, ids=A16, rules=True, **kw):
    r = B._LogitRulesStruct(**kw)
    return L.kvs_process_logits(x, xs, o, os_, dtype, M, V, addr(r) if rules else None, ids, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=(1 << 30) + 1, x=None), B.KVS_ERR_UNSUPPORTED), (dict(M=1 << 30, x=None), B.KVS_ERR_NULL),
    (dict(M=-1), B.KVS_ERR_DIMS), (dict(V=0), B.KVS_ERR_DIMS), (dict(V=(1 << 19) + 1), B.KVS_ERR_UNSUPPORTED),
    (dict(dtype=7), B.KVS_ERR_UNSUPPORTED), (dict(x=None), B.KVS_ERR_NULL), (dict(rules=False), B.KVS_ERR_NULL),
    (dict(o=None, ids=None), B.KVS_ERR_NULL), (dict(xs=999), B.KVS_ERR_DIMS), (dict(os_=999), B.KVS_ERR_DIMS),
    (dict(x=A16 + 2), B.KVS_ERR_ALIGN), (dict(x=A16 + 1, dtype=B.KVS_BF16), B.KVS_ERR_ALIGN),
    (dict(ids=A16 + 2), B.KVS_ERR_ALIGN), (dict(history=A16), B.KVS_ERR_NULL),
    (dict(history=A16, history_offsets=A16, history_len=-1), B.KVS_ERR_DIMS),
    (dict(history=A16, history_offsets=A16, history_len=(1 << 29) + 1), B.KVS_ERR_DIMS),
    (dict(bias_ids=A16, bias_values=A16, bias_offsets=A16, bias_len=-1), B.KVS_ERR_DIMS),
    (dict(bias_ids=A16, bias_values=A16, bias_offsets=A16, bias_len=(1 << 29) + 1), B.KVS_ERR_DIMS),
    (dict(bias_ids=A16, bias_offsets=A16), B.KVS_ERR_NULL), (dict(bias_ids=A16, bias_values=A16), B.KVS_ERR_NULL),
    (dict(mask=A16, mask_count=1), B.KVS_ERR_DIMS), (dict(mask=A16, mask_rows=A16, mask_count=0), B.KVS_ERR_DIMS),
    (dict(repetition=A16 + 2), B.KVS_ERR_ALIGN), (dict(M=0, x=None, o=None, ids=None), B.KVS_OK),
])
def test_process_logits_validation(L, kw, code):
    assert logits(L, **kw) == code


# ---- outputs that overlap inputs ----------------------------------------------------------------
# (The overlap check is the last one.  A call that passes it has no device to run on here; where
# there is one, nothing may be launched at these addresses.)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch at made-up addresses")


def shares_a_byte(a, sa, la, b, sb, lb, n):
    at = set()
    for i in range(n):
        at.update(range(a + i * sa, a + i * sa + la))
    return any(not at.isdisjoint(range(b + j * sb, b + j * sb + lb)) for j in range(n))


@no_gpu
def test_attention_out_over_queries(L):
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(400):
        n = int(rng.integers(1, 7))
        qs, os_ = (int(x) for x in 256 + 4 * rng.integers(0, 80, 2))
        if rng.random() < 0.5:
            os_ = qs
        out = A16 + 16 * int(rng.integers(-900, 900))
        want = shares_a_byte(A16, qs * 4, 1024, out, os_ * 4, 1024, n)
        seen.add((want, qs == os_))
        got = attend(L, cache(), batch(rows=n), qs=qs, out=out, os_=os_)
        assert got == (B.KVS_ERR_OVERLAP if want else B.KVS_ERR_LAUNCH), (n, qs, os_, out - A16)
    assert len(seen) == 4


@no_gpu
@pytest.mark.parametrize("kw,overlap", [
    (dict(o=A16), False), (dict(o=A16, os_=272), True), (dict(o=A16, os_=272, rows=1), False),
    (dict(o=A16 + 16), True), (dict(o=A16 + 1024, qs=512, os_=512), False), (dict(o=A16 + 1008, qs=512, os_=512), True),
    (dict(o=A16 + 5 * 1024), False), (dict(o=A16 + 5 * 1024 - 16), True),
    (dict(k=A16 + 8192, o=A16 + 8192 - 1024, rows=1), False), (dict(k=A16 + 8192, o=A16 + 8192 - 1008, rows=1), True),
    (dict(v=A16 + 8192, o=A16 + 8192 + 512, rows=1), False), (dict(v=A16 + 8192, o=A16 + 8192 + 496, rows=1), True),
])
def test_rope_queries_out(L, kw, overlap):
    far = dict(k=A16 + (1 << 16), v=A16 + (1 << 17))
    rows = kw.pop("rows", 5)
    assert rope(L, cache(), batch(rows=rows), **{**far, **kw}) == \
        (B.KVS_ERR_OVERLAP if overlap else B.KVS_ERR_LAUNCH)


@no_gpu
@pytest.mark.parametrize("kw,overlap", [
    (dict(), False), (dict(os_=1001), True), (dict(os_=1001, M=1), False), (dict(o=A16 + 4), True),
    (dict(o=A16 + 4000, xs=2000, os_=2000), False), (dict(o=A16 + 3996, xs=2000, os_=2000), True),
    (dict(o=A16 + 8000), False), (dict(o=A16 + 7996), True), (dict(o=A16 - 8000), False), (dict(o=None), False),
])
def test_logits_out(L, kw, overlap):
    assert logits(L, **kw) == (B.KVS_ERR_OVERLAP if overlap else B.KVS_ERR_LAUNCH)


# ---- frequency tables -------------------------------------------------------------------------
def table(L, rot, base=10000.0, kind=0, factor=1.0, length=0.0, slow=1.0, fast=32.0):
    out, scale = np.zeros(max(rot // 2, 1), np.float32), ctypes.c_float(-1)
    rc = L.kvs_rope_frequencies(rot, base, kind, factor, length, slow, fast, out.ctypes.data,
                                ctypes.addressof(scale))
    return rc, out.astype(np.float64), scale.value


@pytest.mark.parametrize("rot", [2, 4, 64, 90, 128])
def test_plain_linear_and_ntk_tables(L, rot):
    j = np.arange(rot // 2)
    w = 10000.0 ** (-2.0 * j / rot)
    for kind, factor, want in ((0, 0.0, w), (1, 4.0, w / 4)) + (
            ((2, 8.0, (10000.0 * 8.0 ** (rot / (rot - 2))) ** (-2.0 * j / rot)),) if rot > 2 else ()):
        rc, got, scale = table(L, rot, kind=kind, factor=factor)
        assert rc == 0 and scale == 1.0
        assert np.abs(got / want - 1).max() <= 2.0 ** -23
    if rot > 2:  # the slowest pair is compressed by the factor, the fastest kept
        rc, got, _ = table(L, rot, kind=2, factor=8.0)
        assert abs(got[0] - 1) < 1e-6 and abs(got[-1] / (w[-1] / 8) - 1) < 1e-5


def test_bands_and_yarn_keep_fast_pairs_and_compress_slow_ones(L):
    rot, base, factor, length = 128, 500000.0, 8.0, 8192.0
    j = np.arange(64)
    w = base ** (-2.0 * j / rot)
    turns = length * w / (2 * np.pi)
    rc, got, scale = table(L, rot, base, 4, factor, length, 1.0, 4.0)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert rc == 0 and scale == 1.0
    assert np.abs(got / (keep * w + (1 - keep) * w / factor) - 1).max() < 2.0 ** -22
    assert (keep == 0).any() and (keep == 1).any() and ((keep > 0) & (keep < 1)).any()
    rc, got, scale = table(L, rot, base, 3, factor, length, 1.0, 32.0)
    assert rc == 0 and abs(scale - (0.1 * np.log(8.0) + 1)) < 1e-6
    assert np.abs(got[turns > 40] / w[turns > 40] - 1).max() < 1e-6
    assert np.abs(got[turns < 0.5] / (w[turns < 0.5] / factor) - 1).max() < 1e-6
    ratio = got / w
    assert (np.diff(ratio) <= 1e-6).all() and (ratio >= 1 / factor - 1e-6).all() and (ratio <= 1 + 1e-6).all()


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=-2), dict(rot=64, base=0.0), dict(rot=64, kind=5),
                                dict(rot=64, kind=-1), dict(rot=64, kind=1, factor=0.5), dict(rot=2, kind=2, factor=2.0),
                                dict(rot=64, kind=3, factor=2.0), dict(rot=64, kind=3, factor=2.0, length=10.0, slow=4.0, fast=4.0),
                                dict(rot=64, kind=4, factor=2.0, length=10.0, slow=0.0), dict(rot=64, base=float("nan"))])
def test_frequency_refusals(L, kw):
    assert table(L, **kw)[0] == B.KVS_ERR_DIMS


@pytest.mark.parametrize("kw", [
    dict(base=np.inf), dict(kind=1, factor=np.inf), dict(kind=2, factor=np.inf), dict(kind=3, factor=np.inf, length=100.0),
    dict(kind=3, factor=2.0, length=np.inf), dict(kind=4, factor=2.0, length=np.inf),
    dict(kind=4, factor=2.0, length=100.0, fast=np.inf), dict(base=1e-7), dict(base=1e-300), dict(base=np.inf, kind=3, factor=2.0, length=100.0)])
def test_tables_that_the_rotation_does_not_take(L, kw):
    """Finite entries up to 1e6 are what kvs_rope_scatter_paged asks for."""
    assert table(L, 64, **kw)[0] == B.KVS_ERR_DIMS
    assert table(L, 64, base=1e-6)[0] == 0 and table(L, 64, base=1e-6)[1].max() <= 1e6


@pytest.mark.parametrize("length,slow", [(3.0, 1.0), (6.0, 1.0), (100.0, 20.0), (0.01, 1.0)])
def test_yarn_where_no_pair_turns_the_slow_number_of_times(L, length, slow):
    """Pair 0 turns length / 2 pi times: below `slow` it is compressed like the others."""
    rc, got, _ = table(L, 64, 10000.0, 3, 4.0, length, slow, 32.0)
    want = 10000.0 ** (-2.0 * np.arange(32) / 64) / 4
    assert rc == 0 and np.abs(got / want - 1).max() <= 2.0 ** -23


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_yarn_needs_pairs_of_different_speed(L, base):
    """With base <= 1 no pair is slower than the first, and the ramp over the pairs means nothing."""
    assert table(L, 64, base, 3, 2.0, 100.0)[0] == B.KVS_ERR_DIMS
    assert table(L, 64, base, 4, 2.0, 100.0)[0] == 0


def test_frequency_null(L):
    assert L.kvs_rope_frequencies(64, 1e4, 0, 1.0, 0.0, 1.0, 2.0, None, None) == B.KVS_ERR_NULL
