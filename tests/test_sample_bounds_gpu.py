"""kvs_sample_logits where its blocks work for each other and where its arithmetic ends: rows that
one block of a cluster finishes alone, many of them in flight."""
import pytest
import torch

from paged_helpers import DEV, DTYPES
from split_flash_decoding_kvcachescatter_gb300 import binding as B
from test_sample_gpu import check, logits, uniforms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,V", [(1, 152064), (2, 40001), (37, 152064), (300, 9000)])
@pytest.mark.parametrize("k", [2, 20, 50])
def test_rows_of_a_small_top_k_in_flight_together(dtype, M, V, k):
    """Block 0 of a cluster finishes such a row while the others leave: calls one behind the other,
    on two streams, whose blocks take each other's place on the SMs at once."""
    x = logits(M, V, dtype, seed=k)
    u = uniforms(M, k)
    want = check(x, u, k=[k] * M, p=[0.9] * M)
    uu, kk = torch.tensor(u, device=DEV), torch.full((M,), k, dtype=torch.int32, device=DEV)
    p = torch.full((M,), 0.9, device=DEV)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [torch.full((40, M), -1, dtype=torch.int32, device=DEV) for _ in streams]
    odds = [torch.full((40, M), 7.0, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for i in range(40):
        for s, g, o in zip(streams, got, odds):
            B.kvs_sample_logits(x, uu, token_ids=g[i], top_k=kk, top_p=p, token_probs=o[i], stream=s)
    torch.cuda.synchronize()
    for g, o in zip(got, odds):
        assert torch.equal(g, want.expand(40, M))
        assert torch.equal(o, o[:1].expand(40, M))
