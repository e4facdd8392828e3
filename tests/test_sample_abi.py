"""Host-side refusals of kvs_sample_logits: outputs that lie over inputs or one another."""
import ctypes

import pytest
import torch

from split_flash_decoding_kvcachescatter_gb300 import binding as B
from split_flash_decoding_kvcachescatter_gb300 import build as kbuild

STEP = 1 << 24                        # far apart, never dereferenced (validation fails first)
NAMES = ("logits", "uniforms", "temperature", "top_k", "top_p", "min_p", "token_ids", "token_probs", "probs")
PLACE = {n: STEP * (i + 1) for i, n in enumerate(NAMES)}
M, V = 3, 1000
VECTORS = [n for n in NAMES if n not in ("logits", "probs")]
RULES = ("temperature", "top_k", "top_p", "min_p")


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return B.lib()


def sample(L, m=M, ps=V, xs=V, dtype=B.KVS_F32, **at):
    p = {**PLACE, **at}
    r = ctypes.create_string_buffer(B._pack_sample(*(p[n] or 0 for n in RULES)))
    return L.kvs_sample_logits(p["logits"], xs, dtype, m, V, p["uniforms"], r, p["token_ids"], p["token_probs"],
                               p["probs"], ps, None)


@pytest.mark.parametrize("name", [n for n in NAMES if n != "probs"])
@pytest.mark.parametrize("off", [0, 4 * V, 4 * (M * V - 1)])
def test_probs_over_anything(L, name, off):
    """The first, a later and the last element of the probabilities."""
    assert sample(L, probs=PLACE[name] - off) == B.KVS_ERR_OVERLAP
    # the last element of what they lie over
    last = 4 * ((M * V if name == "logits" else M) - 1)
    assert sample(L, probs=PLACE[name] + last) == B.KVS_ERR_OVERLAP


@pytest.mark.parametrize("out", ["token_ids", "token_probs"])
@pytest.mark.parametrize("name", VECTORS)
@pytest.mark.parametrize("off", [0, 4, 8, -4, -8])
def test_vectors_over_vectors(L, out, name, off):
    if name == out or (name == "uniforms" and off == 0):
        return
    assert sample(L, **{out: PLACE[name] + off}) == B.KVS_ERR_OVERLAP


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch at made-up addresses")
def test_what_lies_beside_passes(L):
    """(There is no device to run on: what passes the checks ends there.)"""
    ok = B.KVS_ERR_LAUNCH
    assert sample(L) == ok
    for out in ("token_ids", "token_probs"):
        assert sample(L, **{out: PLACE["uniforms"]}) == ok  # in place
        for name in VECTORS:
            if name != out:
                assert sample(L, **{out: PLACE[name] + 4 * M}) == ok
                assert sample(L, **{out: PLACE[name] - 4 * M}) == ok
    for name in VECTORS:
        assert sample(L, probs=PLACE[name] + 4 * M) == ok
        assert sample(L, probs=PLACE[name] - 4 * M * V) == ok
        # between two rows of the probabilities
        assert sample(L, probs=PLACE[name] - 4 * V, ps=V + M) == ok
        assert sample(L, probs=PLACE[name] - 4 * V + 4, ps=V + M) == B.KVS_ERR_OVERLAP
    for name in ("token_ids", "token_probs", "probs", *RULES):
        assert sample(L, **{name: None}) == ok
    assert sample(L, m=1, token_ids=PLACE["temperature"] + 4) == ok
