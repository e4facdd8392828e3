"""kvs_process_logits: bit for bit against the rules applied one float32
operation at a time, and against 64 bits; tokens by the argmax rule."""
import numpy as np
import pytest
import torch

import oracle
from paged_helpers import DEV, DTYPES, half_step
from split_flash_decoding_kvcachescatter_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


class Rules:
    def __init__(self, M, V, history=50, bias=5, mask=True, seed=0):
        r = np.random.default_rng(seed)
        self.M, self.V = M, V
        lens = r.integers(0, history + 1, M)
        self.h = [np.where(r.random(n) < 0.5, r.integers(0, min(V, 7), n), r.integers(0, V, n)).astype(np.int32)
                  for n in lens]
        for x in self.h:
            x[r.random(len(x)) < 0.1] = -1  # padding is ignored
        self.prompt = np.array([r.integers(0, n + 1) for n in lens], np.int32)
        self.rep = r.uniform(0.8, 1.5, M).astype(np.float32)
        self.pres = r.uniform(-1, 1, M).astype(np.float32)
        self.freq = r.uniform(-0.2, 0.6, M).astype(np.float32)
        nb = r.integers(0, bias + 1, M) if bias else np.zeros(M, int)
        self.b_ids = [r.integers(-1, min(V, 20), n).astype(np.int32) for n in nb]  # often the same id
        self.b_val = [r.uniform(-5, 5, n).astype(np.float32) for n in nb]
        self.words = None
        if mask:
            self.words = (r.random((max(1, M // 2), (V + 31) // 32 * 32)) < 0.3)
            self.mask_rows = r.integers(-1, len(self.words), M).astype(np.int32)

    def kwargs(self):
        def cat(x, dt):
            return torch.from_numpy(np.concatenate(list(x) + [np.zeros(0, dt)]).astype(dt)).to(DEV)

        def off(x):
            return torch.from_numpy(np.concatenate([[0], np.cumsum([len(a) for a in x])]).astype(np.int32)).to(DEV)
        t = lambda a: torch.from_numpy(a).to(DEV)
        kw = dict(history=cat(self.h, np.int32), history_offsets=off(self.h), prompt_lens=t(self.prompt),
                  repetition=t(self.rep), presence=t(self.pres), frequency=t(self.freq),
                  bias_ids=cat(self.b_ids, np.int32), bias_values=cat(self.b_val, np.float32),
                  bias_offsets=off(self.b_ids))
        if self.words is not None:
            kw["mask"] = t(np.packbits(self.words, axis=1, bitorder="little").view(np.int32).copy())
            kw["mask_rows"] = t(self.mask_rows)
        return kw

    def apply(self, x, ft):
        """The rules on float rows x, every operation in the numpy type ft."""
        x = x.astype(ft)
        for m in range(self.M):
            h = self.h[m]
            ok = (h >= 0) & (h < self.V)
            seen = np.unique(h[ok])
            row = x[m]
            row[seen] = np.where(row[seen] > 0, row[seen] / ft(self.rep[m]), row[seen] * ft(self.rep[m]))
            made, times = np.unique(h[ok & (np.arange(len(h)) >= self.prompt[m])], return_counts=True)
            row[made] = row[made] - ft(self.freq[m]) * times.astype(ft)
            row[made] = row[made] - ft(self.pres[m])
            for i, v in zip(self.b_ids[m], self.b_val[m]):
                if i >= 0:
                    row[i] = row[i] + ft(v)
            if self.words is not None and self.mask_rows[m] >= 0:
                row[~self.words[self.mask_rows[m]][:self.V]] = -np.inf
        return x


def logits(M, V, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (4 * torch.empty(M, V, device=DEV).normal_(generator=g)).to(DTYPES[dtype])


def check(x, out, ids, rules):
    """x: the logits before the call (the kernel's input)."""
    want = torch.from_numpy(rules.apply(x.float().cpu().numpy(), np.float32)).to(x.dtype)
    got = out.cpu()
    assert torch.equal(got.float(), want.float())
    exact = rules.apply(x.double().cpu().numpy(), np.float64)
    # at most 8 operations of a logit in float32, on values under 64, and one rounding to the type
    fin = np.isfinite(exact)
    n_ops = 5 + max([len(b) for b in rules.b_ids] + [0])
    err = np.abs(got.double().numpy()[fin] - exact[fin])
    assert (err <= n_ops * 64 * 2.0 ** -24 + half_step(x.dtype) * (np.abs(exact[fin]) + 1e-3)).all()
    assert np.array_equal(ids.cpu().numpy(), oracle.argmax_rows(np.ascontiguousarray(got.float().numpy())))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,V", [(1, 1), (1, 7), (3, 31), (2, 33), (5, 1000), (4, 32001), (2, 152064), (1, 400003), (200, 129)])
def test_matches_the_rules(dtype, M, V):
    r = Rules(M, V, history=300, bias=20, seed=M * 7 + V)
    x = logits(M, V, dtype, V)
    out, status = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = B.kvs_process_logits(x, out, d_status=status, **r.kwargs())
    assert int(status.item()) == 0
    check(x, out, ids, r)


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_history_of_few_tokens(dtype):
    r = Rules(3, 5000, history=20000, bias=0, mask=False, seed=1)
    x = logits(3, 5000, dtype, 2)
    out = torch.empty_like(x)
    ids = B.kvs_process_logits(x, out, **r.kwargs())
    check(x, out, ids, r)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad_in,pad_out", [(0, 0), (3, 3), (1, 2), (8, 0)])
def test_strides_alignment_and_in_place(dtype, pad_in, pad_out):
    M, V = 5, 2051
    r = Rules(M, V, seed=3)
    wide = torch.full((M, V + pad_in), 9.0, dtype=DTYPES[dtype], device=DEV)
    wide[:, :V] = logits(M, V, dtype, 4)
    x = wide[:, :V]
    out_wide = torch.full((M, V + pad_out), 9.0, dtype=DTYPES[dtype], device=DEV)
    ids = B.kvs_process_logits(x, out_wide[:, :V], **r.kwargs())
    check(x, out_wide[:, :V], ids, r)
    assert (out_wide[:, V:] == 9).all()
    before = x.clone()
    only = B.kvs_process_logits(x, None, **r.kwargs())
    assert torch.equal(x, before) and torch.equal(only, ids)
    ids = B.kvs_process_logits(x, x, **r.kwargs())
    check(before, x, ids, r)
    assert (wide[:, V:] == 9).all()


def test_each_rule_alone_and_none():
    M, V = 4, 3001
    x = logits(M, V, "f32", 5)
    r = Rules(M, V, seed=6)
    kw = r.kwargs()
    out = torch.empty_like(x)
    ids = B.kvs_process_logits(x, out)
    assert torch.equal(out, x) and torch.equal(ids, B.kvs_argmax(x))
    hist = dict(history=kw["history"], history_offsets=kw["history_offsets"])
    one = np.ones(M, np.float32)
    none = dict(rep=one, pres=0 * one, freq=0 * one, b_ids=[np.zeros(0, np.int32)] * M,
                b_val=[np.zeros(0, np.float32)] * M, words=None, prompt=0 * r.prompt)
    for names, keep in ((("repetition",), ("rep",)), (("presence", "prompt_lens"), ("pres", "prompt")),
                        (("frequency",), ("freq",)), (("bias_ids", "bias_values", "bias_offsets"), ("b_ids", "b_val")),
                        (("mask", "mask_rows"), ("words",))):
        alone = Rules(M, V, seed=6)
        for k, v in none.items():
            if k not in keep:
                setattr(alone, k, v)
        ids = B.kvs_process_logits(x, out, **hist, **{k: kw[k] for k in names})
        check(x, out, ids, alone)


def test_values_that_are_not_numbers():
    V = 1000
    x = torch.zeros(5, V, device=DEV)
    x[0] = torch.nan
    x[1] = -torch.inf
    x[2, 5], x[2, 17], x[2, 3] = torch.inf, torch.inf, torch.nan
    x[3, 999] = 1.0
    x[4] = 1.0
    words = np.ones((2, 32 * 32), bool)
    words[0] = False      # a grammar that allows nothing
    words[1, :8] = False
    mask = torch.from_numpy(np.packbits(words, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)
    rows = torch.tensor([-1, -1, 1, 0, 1], dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    ids = B.kvs_process_logits(x, out, mask=mask, mask_rows=rows)
    assert ids.tolist() == [0, 0, 17, 0, 8]
    assert torch.isinf(out[3]).all() and torch.isinf(out[4, :8]).all()
    assert out[0].isnan().all()


def test_bad_lists_count_as_empty_and_are_reported():
    M, V = 3, 600
    x = logits(M, V, "f32", 7)
    for key, code in (("history_offsets", B.KVS_ERR_ROWS), ("bias_offsets", B.KVS_ERR_ROWS), ("mask_rows", B.KVS_ERR_PAGE)):
        r = Rules(M, V, seed=8)
        kw = r.kwargs()
        if key == "mask_rows":
            kw[key][2] = 99
            r.mask_rows[2] = -1
        else:
            kw[key][3] = 10 ** 6  # row 2 ends outside its list
            if key == "history_offsets":
                r.h[2] = r.h[2][:0]
            else:
                r.b_ids[2], r.b_val[2] = r.b_ids[2][:0], r.b_val[2][:0]
        out, status = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device=DEV)
        ids = B.kvs_process_logits(x, out, d_status=status, **kw)
        assert int(status.item()) == code, key
        check(x, out, ids, r)


def test_graph_replay_and_same_bits():
    r = Rules(6, 40000, history=3000, bias=30, seed=9)
    kw = r.kwargs()
    x = logits(6, 40000, "bf16", 10)
    out, ids = torch.empty_like(x), torch.empty(6, dtype=torch.int32, device=DEV)
    B.kvs_process_logits(x, out, token_ids=ids, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kvs_process_logits(x, out, token_ids=ids, **kw)
    for seed in (11, 12):
        x.copy_(logits(6, 40000, "bf16", seed))
        graph.replay()
        torch.cuda.synchronize()
        check(x, out, ids, r)


def test_refusals_of_the_binding():
    x = logits(2, 100, "f32", 13)
    with pytest.raises(TypeError):
        B.kvs_process_logits(x.double())
    with pytest.raises(TypeError):
        B.kvs_process_logits(x.T)
    with pytest.raises(TypeError):
        B.kvs_process_logits(x, torch.empty(2, 99, device=DEV))
    with pytest.raises(ValueError):
        B.kvs_process_logits(x, history=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        B.kvs_process_logits(x, mask=torch.zeros(2, 3, dtype=torch.int32, device=DEV))
    with pytest.raises(B.KvsError) as e:
        B.kvs_process_logits(x, mask=torch.zeros(1, 4, dtype=torch.int32, device=DEV))
    assert e.value.status == B.KVS_ERR_DIMS
    with pytest.raises(TypeError):
        B.kvs_process_logits(x, repetition=torch.ones(3, device=DEV))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,names", [(900, 40), (5000, 1), (40001, 6000), (152064, 152064)])
def test_bias_lists_with_repeated_ids(dtype, V, names):
    """Thousands of entries, most ids many times: the values add up in list order."""
    M = 3
    r = Rules(M, V, history=400, bias=0, seed=V)
    g = np.random.default_rng(names)
    r.b_ids = [g.integers(-1, names, n).astype(np.int32) for n in (4001, 33, 0)]
    r.b_val = [g.uniform(-5, 5, len(i)).astype(np.float32) for i in r.b_ids]
    for i in r.b_ids[:2]:
        i[-1] = i[0] = min(V - 1, 5)  # one at least
    x = logits(M, V, dtype, 20)
    out = torch.empty_like(x)
    ids = B.kvs_process_logits(x, out, **r.kwargs())
    want = torch.from_numpy(r.apply(x.float().cpu().numpy(), np.float32)).to(x.dtype)
    assert torch.equal(out.cpu(), want)
    assert np.array_equal(ids.cpu().numpy(), oracle.argmax_rows(np.ascontiguousarray(want.float().numpy())))
    only = B.kvs_process_logits(x, None, **r.kwargs())
    B.kvs_process_logits(x, x, **r.kwargs())
    assert torch.equal(only, ids) and torch.equal(x, out)


def test_repeated_ids_cost_what_a_list_costs():
    """One id twice in a list of 20,000: no more than a few passes over it."""
    M, V, n = 4, 152064, 20000
    x = logits(M, V, "f32", 21)
    out, took = torch.empty_like(x), []
    for repeat in (False, True):
        r = Rules(M, V, history=10, bias=0, mask=False, seed=22)
        r.b_ids = [np.random.default_rng(m).permutation(V)[:n].astype(np.int32) for m in range(M)]
        r.b_val = [np.ones(n, np.float32)] * M
        if repeat:
            for i in r.b_ids:
                i[n // 2] = i[7]
        kw = r.kwargs()
        ts = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            ids = B.kvs_process_logits(x, out, **kw)
            b.record()
            torch.cuda.synchronize()
            ts.append(a.elapsed_time(b))
        check(x, out, ids, r)
        took.append(min(ts))
    assert took[1] < 10 * took[0] + 0.5, took


@pytest.mark.parametrize("M,V,dtype", [(36, 152064, "f32"), (37, 152064, "bf16"), (75, 32001, "bf16"), (300, 32001, "f16"),
                                       (153, 50000, "f32"), (15, 262144, "bf16"), (3, 2 ** 19, "f32")])
def test_batches_around_the_cluster_rule(M, V, dtype):
    """One row more than are resident at once, words that leave an SM one block, the largest vocabulary."""
    r = Rules(M, V, history=200, bias=4, seed=M)
    x = logits(M, V, dtype, M)
    out = torch.empty_like(x)
    ids = B.kvs_process_logits(x, out, **r.kwargs())
    check(x, out, ids, r)
