"""kvs_sample_logits against the definition in 64 bits: rules alone and together, ties, masked and
infinite logits, vocabularies from one token on, strides, graphs."""
import math

import numpy as np
import pytest
import torch

from paged_helpers import DEV, DTYPES
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


def by_definition(x, u, t=1.0, k=0, p=1.0, least=0.0):
    """(token, probs, margin) of a row in 64 bits; margin: how far the decisions are from borders,
    as a share of the weight."""
    V = len(x)
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    probs = np.zeros(V)
    if not (x > -np.inf).any():
        return 0, probs, 1.0
    order = np.lexsort((np.arange(V), -x))
    order = order[x[order] > -np.inf]
    margin = 1.0
    if not t >= 2.0 ** -126:
        order, w = order[:1], np.ones(1)
    else:
        if k > 0:
            order = order[:k]
        top = x[order[0]]
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            w = np.where(x[order] == top, 1.0, 0.0) if np.isinf(top) else np.exp((x[order] - top) / float(t))
        if p < 1:
            sums = np.cumsum(w)
            need = max(float(p), 0.0) * sums[-1]
            count = max(1, int(np.searchsorted(sums, need)) + 1) if p > 0 else 1
            if p > 0:
                margin = min(margin, float(np.abs(sums - need).min() / sums[-1]))
            order, w = order[:count], w[:count]
        if least > 0:
            cut = min(float(least), 1.0)
            margin = min(margin, float(np.abs(w - cut)[w != cut].min(initial=1.0)))
            order, w = order[w >= cut], w[w >= cut]
    probs[order] = w / w.sum()
    run = np.cumsum(probs)
    u = 0.0 if not u > 0 else min(float(u), 1.0)
    # (before the first kept token the sum is 0, exactly, on both sides)
    margin = min(margin, float(np.abs(run - u)[(run > 0) & (run < run[-1])].min(initial=1.0)))
    last = int(np.flatnonzero(run < run[-1])[-1]) + 1 if (run < run[-1]).any() else 0
    return min(int(np.searchsorted(run, u, side="right")), last), probs, margin


def check(x, u, t=None, k=None, p=None, least=None, **kw):
    """A call with those per-row rules (lists, or None) against the definition of every row."""
    M, V = x.shape
    vec = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device=DEV)  # noqa: E731
    probs = torch.full((M, V), 7.0, device=DEV)
    odds = torch.full((M,), 7.0, device=DEV)
    uu = torch.tensor(u, dtype=torch.float32, device=DEV)
    tt, kk, ppv, ll = vec(t, torch.float32), vec(k, torch.int32), vec(p, torch.float32), vec(least, torch.float32)
    got = B.kvs_sample_logits(x, uu, temperature=tt, top_k=kk, top_p=ppv, min_p=ll, token_probs=odds,
                              probs=probs, **kw)
    alone = B.kvs_sample_logits(x, uu, temperature=tt, top_k=kk, top_p=ppv, min_p=ll)
    assert torch.equal(got, alone)
    host = x.float().cpu().numpy()
    f = lambda v, i, d: d if v is None else v[i].item()  # noqa: E731
    for m in range(M):
        token, want, margin = by_definition(host[m], uu[m].item(), f(tt, m, 1.0), f(kk, m, 0), f(ppv, m, 1.0),
                                            f(ll, m, 0.0))
        assert margin > 1e-11, f"row {m} lies on a border: choose other inputs"
        mine = probs[m].double().cpu().numpy()
        # weights to 2^-40 of themselves (below 2^-45 of the largest: 0), then roundings to float32
        over = np.abs(mine - want) - (want * 2.0 ** -22 + 2.0 ** -44)
        assert (over <= 0).all(), (m, int(over.argmax()), mine[over.argmax()], want[over.argmax()])
        assert ((mine > 0) <= (want > 0)).all(), m
        assert int(got[m]) == token, (m, int(got[m]), token)
        assert odds[m].item() == pytest.approx(want[token], rel=2.0 ** -22, abs=2.0 ** -44)
    return got


def logits(M, V, dtype="f32", seed=0, size=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.empty(M, V, device=DEV).normal_(generator=g) * size).to(DTYPES[dtype])


def uniforms(M, seed=0):
    return np.random.default_rng(seed).random(M, dtype=np.float32).tolist()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 2049, 32001, 152064])
@pytest.mark.parametrize("rules", ["none", "k", "p", "least", "all"])
def test_matches_definition(dtype, V, rules):
    M = 6
    r = np.random.default_rng(V)
    t = r.uniform(0.4, 2.0, M).tolist()
    k = [0, 1, 2, 50, V, 3 * V] if rules in ("k", "all") else None
    p = [0.9, 0.5, 0.99, 1.0, 0.05, 0.999] if rules in ("p", "all") else None
    least = [0.0, 0.02, 0.3, 0.001, 0.9, 0.05] if rules in ("least", "all") else None
    check(logits(M, V, dtype, seed=V), uniforms(M, V), t, k, p, least)


def test_many_draws_of_flat_rows():
    """Nearly equal weights: as many borders as tokens."""
    x = logits(40, 20000, seed=3, size=0.01)
    check(x, uniforms(40, 4))
    check(x, uniforms(40, 5), p=[0.97] * 40)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_lowest_ids(dtype):
    x = logits(5, 5000, dtype, seed=6).mul(2).round().div(2)  # few different values
    check(x, uniforms(5, 7), k=[1, 10, 700, 4999, 33])
    check(x, uniforms(5, 8), p=[0.1, 0.5, 0.9, 0.33, 0.77])
    check(x, uniforms(5, 9), k=[600] * 5, p=[0.5] * 5, least=[0.01] * 5)
    same = torch.full((4, 3001), -3.25, dtype=DTYPES[dtype], device=DEV)
    got = check(same, [0.1234, 0.4321, 0.9, 0.77], k=[0, 17, 1, 2999], p=[1.0, 0.51, 1.0, 0.999])
    assert got.tolist()[2] == 0
    zeros = torch.zeros(2, 777, dtype=DTYPES[dtype], device=DEV)
    zeros[:, ::2] = -0.0  # equal to 0
    check(zeros, [0.3, 0.6], k=[5, 400])


def test_masked_rows_and_infinities():
    inf, nan = math.inf, math.nan
    x = logits(8, 3000, seed=10)
    x[0] = -inf                      # nothing is left
    x[1] = nan
    x[2, 1:] = -inf                  # one token
    x[3, :2999] = -inf
    x[4, ::3] = nan
    x[4, 1::3] = -inf
    x[5, [7, 1234, 2999]] = inf      # those share the row
    x[6] = torch.finfo(torch.float32).min
    x[7, 5:] = torch.finfo(torch.float32).min
    u = [0.5, 0.2, 0.9, 0.1, 0.77, 0.5, 0.4321, 0.6]
    check(x, u)
    check(x, u, k=[5] * 8, p=[0.9] * 8, least=[0.01] * 8)
    odds = torch.full((8,), 7.0, device=DEV)
    ids = B.kvs_sample_logits(x, torch.tensor(u, device=DEV), token_probs=odds)
    assert ids[:4].tolist() == [0, 0, 0, 2999] and odds[:4].tolist() == [0, 0, 1, 1]
    h = torch.full((1, 100), -65504.0, dtype=torch.float16, device=DEV)
    h[0, 50:] = -inf
    check(h, [0.351], p=[0.7])


def test_temperatures():
    x = logits(9, 4000, seed=11)
    t = [0.0, -1.0, math.nan, 1e-30, 1e-45, 0.05, 50.0, 1e30, math.inf]
    got = check(x, uniforms(9, 12), t=t)
    assert torch.equal(got[:5].long(), x[:5].argmax(1))


def test_ends_of_the_rules():
    x = logits(8, 900, seed=13)
    check(x, uniforms(8, 14), p=[0.0, -1.0, 1.0, 2.0, math.nan, float(np.nextafter(np.float32(1), np.float32(0))), 1e-30, 0.3])
    check(x, uniforms(8, 15), k=[-5, 0, 1, 2, 899, 900, 901, 2 ** 31 - 1])
    check(x, uniforms(8, 16), least=[-1.0, 0.0, 1.0, 5.0, 1e-30, 0.999, 0.5, 1e-45])
    for u in (0.0, float(np.nextafter(np.float32(1), np.float32(0)))):
        check(x, [u] * 8, k=[3] * 8)
    # from 1 up the last kept one, below 0 the first
    ids = B.kvs_sample_logits(x, torch.tensor([1.0, 5.0, math.inf, -1.0, -0.0, math.nan, 0.0, 1.0], device=DEV))
    assert ids.tolist() == [899, 899, 899, 0, 0, 0, 0, 899]


def test_strided_rows_and_every_alignment():
    for dtype in DTYPES:
        base = logits(3, 5100, dtype, seed=17)
        for off in range(0, 9):
            check(base[:, off:off + 4321], uniforms(3, off), t=[0.8] * 3, k=[0, 100, 7], p=[0.9, 1.0, 0.6])


def test_probs_with_strides():
    x = logits(3, 1000, seed=18)
    wide = torch.full((3, 2500), 7.0, device=DEV)
    B.kvs_sample_logits(x, torch.tensor([0.1, 0.2, 0.3], device=DEV), probs=wide[:, 700:1700])
    assert torch.allclose(wide[:, 700:1700], torch.softmax(x, 1), rtol=1e-5, atol=0)
    assert (wide[:, :700] == 7).all() and (wide[:, 1700:] == 7).all()


def test_more_rows_than_fit_at_once():
    x = logits(700, 3000, "bf16", seed=19)
    check(x, uniforms(700, 20), k=[30] * 700, p=[0.8] * 700)


def test_frequencies():
    """Even random numbers draw each token as often as its weight says: with u = (i + 1/2) / n a
    token of weight w comes w n times, one more or less at each of its two borders."""
    n = 4096
    x = logits(1, 50, seed=21).expand(n, 50).contiguous()
    u = (torch.arange(n, device=DEV) + 0.5) / n
    ids = B.kvs_sample_logits(x, u, temperature=torch.full((n,), 0.7, device=DEV))
    want = torch.softmax(x[0].double() / 0.7, 0) * n
    assert (torch.bincount(ids.long(), minlength=50) - want).abs().max() < 1


def test_captured_call_follows_its_inputs():
    x = logits(4, 20000, seed=22)
    u = torch.tensor(uniforms(4, 23), device=DEV)
    k = torch.tensor([0, 40, 1, 300], dtype=torch.int32, device=DEV)
    ids = torch.empty(4, dtype=torch.int32, device=DEV)
    B.kvs_sample_logits(x, u, token_ids=ids, top_k=k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.kvs_sample_logits(x, u, token_ids=ids, top_k=k)
    x.copy_(logits(4, 20000, seed=24))
    u.copy_(torch.tensor(uniforms(4, 25)))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, B.kvs_sample_logits(x, u, top_k=k))


def test_after_the_logit_rules():
    """The serving path: rules and a grammar mask, then a draw among what they leave."""
    x = logits(3, 4000, seed=26)
    mask = torch.zeros(3, 125, dtype=torch.int32, device=DEV)
    mask[0, 3], mask[1, 124], mask[2, 0] = 0b1011, -1, 1
    out = torch.empty_like(x)
    B.kvs_process_logits(x, out, mask=mask)
    got = check(out, uniforms(3, 27), p=[0.95] * 3)
    allowed = [{96, 97, 99}, set(range(3968, 4000)), {0}]
    assert all(int(t) in s for t, s in zip(got, allowed))


def test_binding_refuses_wrong_tensors():
    x, u = logits(2, 100), torch.zeros(2, device=DEV)
    for bad in (dict(logits=x.double()), dict(logits=x[0]), dict(uniforms=u[:1]), dict(uniforms=u.double()),
                dict(top_k=torch.zeros(2, device=DEV)), dict(top_p=torch.zeros(3, device=DEV)),
                dict(token_ids=torch.zeros(2, dtype=torch.int64, device=DEV)), dict(probs=torch.zeros(2, 99, device=DEV)),
                dict(logits=x.t())):
        with pytest.raises(TypeError):
            B.kvs_sample_logits(**{**dict(logits=x, uniforms=u), **bad})
    with pytest.raises(B.KvsError):
        B.kvs_sample_logits(x, u, probs=x)
