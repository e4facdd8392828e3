"""The 8-bit cache at the ends of what its scales may be: V scales as far apart as the format allows
under every kernel, infinities, NaN and the largest numbers in appended rows, old scales of any value."""
import math

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES, least_step, within
from q8_helpers import BLOCK, E4M3, e4m3, scale_of
from split_flash_decoding_kvcachescatter_gb300 import binding as B
from test_q8_edges_gpu import KINDS, kind
from test_rope_q8_gpu import Append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


def set_value_scales(b, pick):
    """Gives every live block of V the scale pick(sequence, block, kv head) instead of its own."""
    for i, v in enumerate(b.v):
        L = v.shape[1]
        for j in range(-(-L // BLOCK)):
            at, of_page = int(b.table_host[i, j * BLOCK // b.page]), j * BLOCK % b.page // BLOCK
            for h in range(b.Hkv):
                s = pick(i, j, h)
                part = v[h, j * BLOCK:(j + 1) * BLOCK]
                part *= s / float(b.v_scales[at, h, of_page])
                b.v_scales[at, h, of_page] = s


def check(b, where):
    """b.check(), where a sequence's values may all be 0: its bound is not defined by their size, and
    scales below 2^-60 count as 2^-60, so its outputs are 448 2^-60 at most."""
    got = b.attend()
    ref, bound = b.reference()
    assert int(b.status.item()) == 0, where
    within(got, ref, torch.nan_to_num(bound, nan=448 * 2.0 ** -60 + least_step(b.dtype)), where)


# (smallest scale, largest): 16-bit floats end at 65504, so float16 outputs leave room for 2^6 x 448
SPANS = {"zero and largest": (0.0, 100), "least and largest": (2.0 ** -60, 100), "2^130": (2.0 ** -60, 70)}


@pytest.mark.parametrize("span", SPANS)
@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("order", ["mixed", "small first", "large first"])
def test_keys_under_small_value_scales_keep_their_share(name, span, order):
    """Keys whose values are nothing beside the others' count in the sum of the weights all the same,
    whichever of them comes first."""
    b = kind(name, seed=3)
    least, top = SPANS[span]
    top = 2.0 ** (6 if KINDS[name]["dtype"] == "f16" else top)
    rng = np.random.default_rng(7)
    half = [max(1, -(-v.shape[1] // BLOCK) // 2) for v in b.v]
    def pick(i, j, h):  # noqa: E306
        small = rng.random() < 0.5 if order == "mixed" else (j < half[i]) == (order == "small first")
        return least if small else top
    set_value_scales(b, pick)
    check(b, f"{name}, {span}, {order}")


@pytest.mark.parametrize("name", KINDS)
def test_value_scales_all_over_their_range(name):
    b = kind(name, seed=4)
    top = 6 if KINDS[name]["dtype"] == "f16" else 100
    rng = np.random.default_rng(8)
    set_value_scales(b, lambda i, j, h: 2.0 ** int(rng.integers(-60, top + 1)))
    check(b, name)


# heads that turn whole, in interleaved pairs, not at all (one kernel) and in part (the other one)
LAYOUTS = {"whole": (64, False), "pairs": (64, True), "none": (0, False), "part": (32, False), "odd": (20, False)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_infinities_and_nan_do_not_move_scales(dtype, layout):
    """With an element that is infinite or NaN every scale and every other number are those of the
    same rows with a 0 there; it becomes the largest number, or stays NaN."""
    rot, il = LAYOUTS[layout]
    n, p = [40, 1, 1, 17], [3, 9, 16, 31]
    a, b = (Append(n, p, 8, 2, 64, dtype, 32, rot=rot, interleaved=il, seed=31) for _ in range(2))
    row = [0, 5, 20, 40, 41, 50]  # rows of both directions, of a block with older rows, and alone
    odd = [math.inf, -math.inf, math.nan, math.inf, -math.inf, math.nan]
    at = 63 if rot < 64 else 3
    partner = at if rot < 64 else at - 1 if il else at + 32  # (turned with it)
    for r, x in zip(row, odd):
        a.k[r, :, at], a.v[r, :, at] = x, x
        b.k[r, :, at], b.v[r, :, at] = 0, 0
        a.k[r, :, partner] = x  # both of a pair, so that both of b's are 0
        b.k[r, :, partner] = 0
    a.run()
    b.run()
    position = np.concatenate([np.arange(u, u + m) for m, u in zip(n, p)])
    owner = np.repeat(np.arange(len(n)), n)
    for kv in range(2):
        assert torch.equal(a.scales[kv], b.scales[kv])
        got, want = (x.pages[kv].view(torch.uint8).clone() for x in (a, b))
        for r, x in zip(row, odd):
            page, slot = int(a.table[owner[r], position[r] // 32]), int(position[r] % 32)
            for e in {at, partner} if kv == 0 else {at}:
                there = a.pages[kv][page, :, slot, e].float()
                if kv == 1 or rot < 64:
                    assert torch.isnan(there).all() if math.isnan(x) else (there == math.copysign(448, x)).all()
                else:  # (a turned infinity is infinite or NaN)
                    assert (torch.isnan(there) | (there.abs() == 448)).all()
                got[page, :, slot, e] = want[page, :, slot, e] = 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["whole", "none", "part"])
def test_largest_rows_stay_in_the_range_that_is_read(dtype, layout):
    """Scales end at 2^100; what is larger than 448 2^100 becomes that, and is read as that."""
    rot, il = LAYOUTS[layout]
    a = Append([20, 1], [0, 17], 8, 2, 64, dtype, 16, rot=rot, interleaved=il, seed=32)
    a.k[:] = 0
    a.q[:] = 0
    a.v[:] = 2.0 ** 126
    a.v[3:7] = -2.0 ** 90
    a.run()
    first = a.table[0, :2].tolist()
    assert (a.scales[1][first] == 2.0 ** 100).all() and (a.scales[0][first] == 2.0 ** -60).all()
    v = a.pages[1][first].float().transpose(0, 1).reshape(2, 32, 64)[:, :20]
    assert (v[:, :3] == 448).all() and (v[:, 7:] == 448).all() and (v[:, 3:7] == -2.0 ** -9 * 0).all()
    # the second sequence has older rows under small scales: they become 0
    at = int(a.table[1, 1])
    assert (a.scales[1][at, :, 0] == 2.0 ** 100).all() and (a.pages[1][at, :, 0].float() == 0).all()
    q = torch.zeros(21, 8, 64, dtype=a.dtype, device=DEV)
    out, cache = torch.empty_like(q), a.cache()
    B.kvs_paged_attention_q8(q, cache, a.batch, out, d_status=a.status,
                             workspace=B.paged_attention_q8_workspace(cache, a.batch, 8))
    # even weights: the mean of 448 2^100 over the rows but four of them
    t = torch.arange(20, device=DEV)
    share = 1 - ((t - 2).clamp(0, 4).double() / (t + 1))
    want = 448 * 2.0 ** 100 * share
    assert ((out[:20].double() - want[:, None, None]).abs() <= want[:, None, None] * (
        torch.finfo(a.dtype).eps / 2 + 2.0 ** -11)).all()
    assert int(a.status.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["none", "part"])
@pytest.mark.parametrize("power", [-4, 1])
def test_old_scales_of_any_value(dtype, layout, power):
    """New rows under an old scale that is no power of two go by its reciprocal; where the scale
    grows, the older numbers go by the quotient.  (2^-4: most scales stay, 2^1: most grow.)"""
    rot, il = LAYOUTS[layout]
    a = Append([5, 1, 9], [3, 9, 22], 8, 2, 64, dtype, 16, rot=rot, interleaved=il, seed=33, size=2.0 ** power)
    g = torch.Generator(device=DEV).manual_seed(5)
    for x in a.scales:
        x.mul_(1 + torch.rand(x.shape, generator=g, device=DEV))
    before = [x.clone() for x in a.pages], [x.clone() for x in a.scales]
    a.run()
    stayed = grew = 0
    for i, (n, p) in enumerate(zip(a.n, a.p)):
        count = min(n, BLOCK - p % BLOCK)  # the rows that join older ones
        at, lo = int(a.table[i, p // 16]), p % 16
        r = int(a.offsets[i])
        for kv, src in ((0, a.k), (1, a.v)):
            rows = src[r:r + count, :, rot if kv == 0 else 0:].float().transpose(0, 1)  # (what does not turn)
            off = rot if kv == 0 else 0
            old = before[1][kv][at, :, 0]
            new = a.scales[kv][at, :, 0]
            if kv == 1:  # (turned elements of k may be the largest)
                s = scale_of(rows.double().abs().amax((1, 2))).float()
                assert torch.equal(new, torch.maximum(s, old))
            stayed += int((new == old).sum())
            grew += int((new != old).sum())
            inv = 1 / new  # (float32, correctly rounded)
            want = e4m3((rows * inv[:, None, None]).double())
            assert torch.equal(a.pages[kv][at, :, lo:lo + count, off:].double(), want)
            older, was = a.pages[kv][at, :, :lo].double(), before[0][kv][at, :, :lo]
            ratio = (old / new)[:, None, None]
            want = torch.where(ratio == 1, was.double(), e4m3((was.float() * ratio).double()))
            assert torch.equal(older, want)
    assert (stayed if power < 0 else grew) > 0
