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


def tail_rows(V, low, high, seed, M):
    """One token of weight 1 behind V - 1 others of weights 2^-high to 2^-low, their exact weights."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    e = low + (high - low) * torch.rand(V, generator=g, device=DEV, dtype=torch.float64)
    x = (-e * 0.6931471805599453).float()
    x[V - 1] = 0.0
    return x.expand(M, V).contiguous(), torch.exp(x.double())


@pytest.mark.parametrize("V", [4097, 152064, 2 ** 19])
@pytest.mark.parametrize("low,high", [(40, 46), (44.4, 44.4), (45.2, 45.2), (30, 46)])
def test_long_tails_of_the_smallest_weights(V, low, high):
    """A weight is off by 2^-37 of itself and 2^-45 of the largest, so borders between tokens are by
    2^-36 + V 2^-44 and probabilities by what follows; many weights near the end all at once."""
    M = 96
    x, w = tail_rows(V, low, high, 51, M)
    run = torch.cumsum(w, 0)
    total = run[-1]
    # random numbers within the tail, and some behind it
    u = (torch.rand(M, generator=torch.Generator().manual_seed(52), dtype=torch.float64).to(DEV) * 1.25 *
         (run[-2] / total)).float()
    probs, odds = torch.empty(M, V, device=DEV), torch.empty(M, device=DEV)
    ids = B.kvs_sample_logits(x, u, token_probs=odds, probs=probs).long()
    eps = 2.0 ** -36 + V * 2.0 ** -44
    below = torch.where(ids > 0, run[(ids - 1).clamp_min(0)], 0) / total
    assert (below - eps <= u.double()).all() and (u.double() <= run[ids] / total + eps).all()
    want = (w / total).expand(M, V)
    err = want * (2.0 ** -24 + 2.0 ** -35) + 2.0 ** -45 * (1 + V * want)
    assert ((probs.double() - want).abs() <= err).all()
    assert torch.equal(odds, probs.gather(1, ids[:, None])[:, 0])


@pytest.mark.parametrize("V", [4097, 152064])
def test_min_p_near_the_end_of_the_weights(V):
    M = 4
    x, w = tail_rows(V, 40, 46, 53, M)
    least = torch.tensor([2.0 ** -41, 2.0 ** -43.5, 2.0 ** -44, 2.0 ** -45], device=DEV)
    probs = torch.empty(M, V, device=DEV)
    B.kvs_sample_logits(x, torch.zeros(M, device=DEV), min_p=least, probs=probs)
    for m in range(M):
        slack = w * 2.0 ** -37 + 2.0 ** -45
        kept = probs[m] > 0
        cut = float(least[m])
        assert kept[w - slack > cut].all() and not kept[w + slack < cut].any()


def test_top_p_over_a_tail_near_the_end_of_the_weights():
    """The shortest run from the front, within what the sums of a large vocabulary may be off."""
    V = 2 ** 19
    x, w = tail_rows(V, 40, 46, 54, 3)
    order = torch.argsort(x[0], descending=True, stable=True)
    run = torch.cumsum(w[order], 0)
    share = (run[[V // 5, V // 2, V - 1000]] / run[-1]).float().clamp_max(1 - 2.0 ** -24)
    probs = torch.empty(3, V, device=DEV)
    B.kvs_sample_logits(x, torch.zeros(3, device=DEV), top_p=share, probs=probs)
    eps = 2.0 ** -36 + V * 2.0 ** -44
    for m in range(3):
        kept = probs[m, order] > 0
        n, p = int(kept.sum()), float(share[m])
        assert p < 1 and kept[:n].all()
        assert run[n - 1] / run[-1] >= p - eps and (n == 1 or run[n - 2] / run[-1] < p + eps)
