"""kvs_paged_attention under limits that see a single lost tile of keys and a float32 product
without its low parts; keys whose weights are not alike; bad rows in every kernel."""
import pytest
import torch

from paged_helpers import DEV, DTYPES, Paged, half_step, within
from paged_norms import check_norms
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu

WIDE = 2 ** 19  # room for so many keys a sequence: decode steps take the kernel for long caches


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,p,H,Hkv,D,columns", [
    ([1, 1, 1], [20011, 15000, 5003], 16, 8, 64, WIDE // 64),
    ([1], [40000], 16, 8, 64, WIDE // 64),
    ([2, 0, 1], [31000, 5, 12345], 16, 8, 64, WIDE // 64),
    ([1] * 40, [900 + 7 * i for i in range(40)], 16, 8, 64, 2),
    ([1, 1, 1], [20011, 15000, 5003], 32, 8, 128, WIDE // 64),
    ([1] * 5, [9000, 0, 63, 700, 2999], 40, 8, 128, 2),
    ([1, 2, 1], [1023, 400, 7], 8, 2, 128, 2)])
def test_decode(dtype, n, p, H, Hkv, D, columns):
    b = Paged(n, p, H, Hkv, D, dtype, 64, seed=sum(n) + D, columns=columns)
    check_norms(b, b.attend())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,D", [(14, 2, 64), (32, 8, 128)])
def test_chunks(dtype, H, Hkv, D):
    for n, p, page in (([300, 1, 90], [3300, 8000, 0], 64), ([130, 1, 17], [200, 63, 4000], 16)):
        b = Paged(n, p, H, Hkv, D, dtype, page, seed=sum(n) + D)
        check_norms(b, b.attend(), f"{n}")


def needles(b, at):
    """q of (row, head) along the key at(i, t, h) of its sequence, so that this key takes about
    half of the weight (16,000 to 40,000 others the rest)."""
    G = b.H // b.Hkv
    for i, n in enumerate(b.n):
        a = int(b.offsets_host[i])
        for t in range(n):
            j = torch.tensor([at(i, t, h) for h in range(b.H)], device=DEV)
            g = torch.arange(b.H, device=DEV) // G
            b.q[a + t] = (1.5 * b.k[i][g, j].float()).to(b.dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_tile_of_a_long_cache_counts(dtype):
    """Each 32-key tile of each sequence has a key that some head looks for; first and last keys
    of tiles in turn."""
    p = [20011, 15000, 16383]
    b = Paged([1, 1, 1], p, 64, 8, 64, dtype, 64, seed=31, columns=WIDE // 64)
    for call in range(-(-(max(p) + 1) // (32 * 64))):
        needles(b, lambda i, t, h: min(p[i], (call * 64 + h) * 32 + 31 * (h % 2)))
        check_norms(b, b.attend(), f"call {call}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_tile_of_a_chunk_counts(dtype):
    n, p = [40, 9], [8000, 5001]
    b = Paged(n, p, 32, 8, 64, dtype, 32, seed=32)
    needles(b, lambda i, t, h: min(p[i] + t, (t * 7 + h) * 128 % (p[i] + t) + 127 * (h % 2)))
    check_norms(b, b.attend())


FORMS = {"cluster": ([3, 2, 4], 2), "ranges": ([3, 2, 4], WIDE // 32), "chunk": ([70, 2, 40], 2)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_row_offsets_leave_their_rows_alone(dtype, form):
    n, columns = FORMS[form]
    for at, value in ((1, -1), (2, 1), (3, 1000), (0, -5)):
        b = Paged(n, [30, 20, 10], 8, 2, 64, dtype, 32, seed=33, columns=columns)
        b.row_offsets[at] = value
        out = b.attend()
        assert int(b.status.item()) == B.KVS_ERR_ROWS
        o = b.row_offsets.tolist()
        ref, bound = b.reference()
        for i in range(3):
            a, e = int(b.offsets_host[i]), int(b.offsets_host[i + 1])
            if 0 <= o[i] <= o[i + 1] <= b.rows and o[i + 1] - o[i] <= max(n):
                assert (o[i], o[i + 1]) == (a, e)
                within(out[a:e], ref[a:e], bound[a:e], f"{at} {value} {i}")
            else:
                assert (out[a:e] == 7).all(), (at, value, i)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_positions_mark_their_rows(dtype, form):
    n, columns = FORMS[form]
    for bad in (-1, 2 ** 31 - 1):
        b = Paged(n, [300, 200, 100], 8, 2, 64, dtype, 32, seed=34, columns=columns)
        b.positions[1] = bad
        out = b.attend()
        assert int(b.status.item()) == B.KVS_ERR_POSITION
        ref, bound = b.reference()
        a, e = n[0], n[0] + n[1]
        assert out[a:e].isnan().all()
        keep = [r for r in range(sum(n)) if not a <= r < e]
        within(out[keep], ref[keep], bound[keep], f"{bad}")
