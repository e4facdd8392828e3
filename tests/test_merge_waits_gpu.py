"""The persistent decode kernel's join of a split (sequence, kv head) when waits run out around it:
some warps of a block then find a barrier's phase complete and go on to the join while another one's
wait has just run out and it leaves.  Every call ends, and the next one is right."""
import numpy as np
import pytest
import torch

from split_flash_decoding_kvcachescatter_gb300 import binding as B
from split_flash_decoding_kvcachescatter_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from split_flash_decoding_kvcachescatter_gb300 import build
    build.build()
    B.lib()


@pytest.fixture(autouse=True)
def _restore():
    prev = B.kvs_get_schedule()
    yield
    torch.cuda.synchronize()
    B.kvs_set_wait_limit_ns(B.KVS_WAIT_LIMIT_DEFAULT_NS)
    B.kvs_set_schedule(prev)


@pytest.mark.parametrize("M,H,Hkv,D,L", [(1, 32, 8, 128, 4096), (8, 32, 8, 128, 2048), (4, 14, 2, 64, 2048),
                                         (2, 8, 1, 64, 8000)])
def test_every_call_ends_whatever_wait_runs_out(M, H, Hkv, D, L):
    B.kvs_set_schedule(B.KVS_SCHEDULE_PERSISTENT)
    w = W.custom(positions="uniform", seed=M + D, M=M, num_heads=H, num_kv_heads=Hkv, head_dim=D,
                 max_len=L, chunk_size=0)
    t = W.upload(W.make_inputs(w), w, DEV)
    ws = B.workspace(M, H, Hkv, D, L, 0, device=DEV).fill_(0xFF)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        out = torch.full((M, H, D), 7.0, device=DEV)
        status.zero_()
        B.kvs_decode_step(t["q"], t["k_rows"], t["v_rows"], t["positions"], t["k_cache"], t["v_cache"], out,
                          chunk_size=0, workspace=ws, d_status=status)
        torch.cuda.synchronize()
        return out, int(status.item())

    want, code = step()
    assert code == 0
    seen = set()
    for limit in np.random.default_rng(L).integers(0, 25000, 250).tolist():
        B.kvs_set_wait_limit_ns(limit)
        _, code = step()
        assert code in (B.KVS_OK, B.KVS_ERR_TIMEOUT), limit
        seen.add(code)
        B.kvs_set_wait_limit_ns(B.KVS_WAIT_LIMIT_DEFAULT_NS)
        out, code = step()
        assert code == 0, limit
        assert torch.equal(out, want), limit
    assert B.KVS_ERR_TIMEOUT in seen
