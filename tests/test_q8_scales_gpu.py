"""The 8-bit cache at the ends of what its scales may be: V scales as far apart as the format allows
under every kernel, infinities, NaN and the largest numbers in appended rows, old scales of any value."""
import math

import numpy as np
import pytest
import torch

from paged_helpers import DEV, least_step, within
from q8_helpers import BLOCK
from split_flash_decoding_kvcachescatter_gb300 import binding as B
from test_q8_edges_gpu import KINDS, kind

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
