"""Softmax weights of kvs_paged_attention far below the largest one: many of them still count."""
import pytest
import torch

from paged_helpers import DEV, Paged, within
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


# a cluster a unit, ranges over a long cache, a chunk
@pytest.mark.parametrize("n,p,columns", [(1, 20000, 2), (1, 131071, 2), (40, 131000, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("first", [True, False])
def test_a_long_tail_of_small_weights(n, p, columns, dtype, first):
    """One key has weight 1, the others 2^-26 each (in 16 bits: nothing, if rounded as they are).
    V is 1 at the others: the output is their share of the sum."""
    b = Paged([n], [p], 8, 8, 64, dtype, 64, seed=1, columns=columns)
    L = n + p
    top = 0 if first else p  # (a key that every row attends)
    b.q.zero_()
    b.q[..., 0] = 8
    k = torch.zeros(8, L, 64, dtype=b.dtype, device=DEV)
    k[..., 0] = -8.0
    k[:, top, 0] = 10.0
    v = torch.ones_like(k)
    v[:, top] = 0
    for j in range(-(-L // 64)):
        a, e = 64 * j, min(L, 64 * j + 64)
        b.k_pages[b.table_host[0, j], :, :e - a] = k[:, a:e]
        b.v_pages[b.table_host[0, j], :, :e - a] = v[:, a:e]
    out = b.attend()
    assert int(b.status.item()) == 0
    w = torch.exp(torch.tensor(-18.0, dtype=torch.float64))
    tail = w * (p + torch.arange(n, dtype=torch.float64))
    want = (tail / (1 + tail)).to(DEV)[:, None, None]
    # each weight, each output: one rounding to the type (2^-8, 2^-11); the exponent of 18 and
    # the sums of 131,072 terms in float32: under 2^-10
    rel = 2 * torch.finfo(b.dtype).eps / 2 + 2.0 ** -10
    within(out, want.expand_as(out).contiguous(), rel * want)


@pytest.mark.parametrize("n,p,columns", [(1, 300, 2), (1, 300, 2 ** 13), (40, 300, 2)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_key_far_above_the_others(n, p, columns, dtype):
    """Scores of 8 million and 45 million, where float32 is 1 to 4 apart: the key's value comes out,
    but for its weight's rounding and the output's."""
    for size in (1000.0, 2368.0):
        b = Paged([n], [p], 8, 8, 64, dtype, 64, seed=2, columns=columns)
        b.q.fill_(size)
        b.k_pages.zero_()
        b.v_pages.fill_(1)
        page, slot = int(b.table_host[0, 2]), 7
        b.k_pages[page, :, slot] = size
        b.v_pages[page, :, slot] = -0.75
        out = b.attend()
        assert int(b.status.item()) == 0
        rel = torch.finfo(b.dtype).eps + 2.0 ** -20
        assert ((out.double() + 0.75).abs() <= 0.75 * rel).all(), (size, float(out.min()), float(out.max()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("p,columns", [(900, 2), (5000, 2), (5000, 2 ** 13)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_steps_hold_their_weights_in_more_than_16_bits(p, columns, dtype, D):
    """The output is the definition's, rounded once, but where float32's errors carry it over the
    middle of two numbers: they are under 2^-16 of it, a hundredth of such numbers' distance in
    float16.  With weights rounded to 16 bits a quarter of the elements differ."""
    b = Paged([1] * 4, [p, p - 77, p // 2, 300], 16, 4, D, dtype, 64, seed=D, columns=columns)
    out = b.attend()
    want, _ = b.reference()
    assert float((out == want.to(b.dtype)).double().mean()) > 0.95
