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


@pytest.mark.parametrize("M", [1, 5, 700])
def test_a_row_s_result_in_its_random_number_s_place(M):
    x = logits(M, 9000, seed=41)
    k = torch.tensor([(0, 30, 1)[m % 3] for m in range(M)], dtype=torch.int32, device=DEV)
    u = torch.tensor(uniforms(M, 42), device=DEV)
    odds = torch.empty(M, device=DEV)
    want = B.kvs_sample_logits(x, u, top_k=k, token_probs=odds)
    a, b = u.clone(), u.clone()
    B.kvs_sample_logits(x, a, token_ids=a.view(torch.int32), top_k=k)
    assert torch.equal(a.view(torch.int32), want)
    got = B.kvs_sample_logits(x, b, top_k=k, token_probs=b)
    assert torch.equal(got, want) and torch.equal(b, odds)


def test_the_binding_refuses_results_over_logits():
    wide = torch.zeros(4, 128, device=DEV)
    x, u = wide[:, :100], torch.zeros(4, device=DEV)
    flat = wide.view(-1)
    for at in (0, 3, 97, 128, 3 * 128 + 99):  # the first, a row's end, the next row, the last element
        with pytest.raises(ValueError, match="logits"):
            B.kvs_sample_logits(x, u, token_ids=flat[at:at + 4].view(torch.int32))
        with pytest.raises(ValueError, match="logits"):
            B.kvs_sample_logits(x, u, token_probs=flat[at:at + 4])
    for at in (100, 124, 3 * 128 + 100):  # behind a row
        assert B.kvs_sample_logits(x, u, token_ids=flat[at:at + 4].view(torch.int32)).tolist() == [0] * 4
    for other in ("uniforms", "temperature", "top_p", "min_p"):
        v = torch.full((5,), 0.5, device=DEV)
        with pytest.raises(B.KvsError):
            B.kvs_sample_logits(**{**dict(logits=x, uniforms=u), other: v[:4]}, token_probs=v[1:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [50, 5000, 152064])
def test_a_token_s_probability_is_one_number(dtype, V):
    """The token's probability, the one of its place among all, and that of the call without all."""
    M = 64
    x = logits(M, V, dtype, seed=43)
    u = torch.tensor(uniforms(M, 44), device=DEV)
    k = torch.tensor([(0, 50, 7, 400)[m % 4] for m in range(M)], dtype=torch.int32, device=DEV)
    p = torch.tensor([(1.0, 0.9)[m // 4 % 2] for m in range(M)], device=DEV)
    odds, alone, probs = (torch.empty(M, device=DEV), torch.empty(M, device=DEV), torch.empty(M, V, device=DEV))
    ids = B.kvs_sample_logits(x, u, top_k=k, top_p=p, token_probs=odds, probs=probs)
    B.kvs_sample_logits(x, u, top_k=k, top_p=p, token_probs=alone)
    assert torch.equal(odds, probs.gather(1, ids.long()[:, None])[:, 0])
    assert torch.equal(odds, alone)
    # one rounding to float32: weights are off by 2^-37 of themselves and 2^-45 of the largest, of
    # which the sum has at most that many, and all of it once more for the sum
    host = x.double()
    order = torch.argsort(host, dim=1, descending=True, stable=True)
    w = torch.exp(host - host.amax(1, keepdim=True))
    kk = torch.where(k > 0, k, V).long()
    rank = torch.empty_like(order).scatter_(1, order, torch.arange(V, device=DEV).expand(M, V))
    w = torch.where(rank < kk[:, None], w, 0)
    plain = p == 1
    want = (w / w.sum(1, keepdim=True))[plain]
    over = (probs[plain].double() - want).abs() - want * (2.0 ** -24 + 2.0 ** -35) - 2.0 ** -45 * (1 + V * want)
    assert (over <= 0).all()
