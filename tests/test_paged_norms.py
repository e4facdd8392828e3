"""The limits that the long-cache tests use, shown on the CPU to see what they are for: one tile
of keys left out, and float32 products without their low parts."""
import pytest
import torch

from paged_helpers import DTYPES
from paged_norms import attention64, norm_limit, weight_rounding, worst


def inputs(n, L, H, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(dtype) for s in ((n, H, D), (Hkv, L, D), (Hkv, L, D))]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("L", [9001, 20012, 40001])
def test_a_lost_tile_is_outside(dtype, L):
    dt = DTYPES[dtype]
    q, k, v = inputs(1, L, 4, 2, 64, dt, L)
    o, spread, size = attention64(q, k, v, L - 1)
    limit = norm_limit(o, spread, size, L, dt, weight_rounding(dt, False))
    for tile in range(5, L // 32, L // 32 // 12):
        part, _, _ = attention64(q, k, v, L - 1, lost=slice(32 * tile, 32 * tile + 32))
        err = (part - o).norm(dim=-1) / limit
        assert float(err.min()) > 1.5, (tile, err)  # (any rounding on top is within `limit` itself)


@pytest.mark.parametrize("n,L,D", [(1, 700, 64), (1, 20012, 64), (1, 9001, 128), (100, 2000, 64), (100, 2000, 128)])
def test_one_tf32_product_is_outside(n, L, D):
    q, k, v = inputs(n, L, 4, 2, D, torch.float32, L + D)
    o, spread, size = attention64(q, k, v, L - n)
    limit = norm_limit(o, spread, size, L, torch.float32, 0.0)
    rough, _, _ = attention64(q, k, v, L - n, q_low=False)
    assert worst(rough, o, limit) > 2
