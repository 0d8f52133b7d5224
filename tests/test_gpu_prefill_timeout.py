"""The bounded waits inside the prefill kernels, made to expire without a
fault: the test hook leaves the tensor-core warp idle, so the others wait for
scores that never come.  The launch records PKV_ERR_TIMEOUT and stores no row,
nothing is in flight when it ends, and the next call is right."""
import pytest
import torch

import oracle
import pkv_workloads as W
from gpu_helpers import DeviceStep, assert_close
from scaled_batch import Batch, bf16_rows
from test_gpu_scaled_attention import KINDS, check, pkv, prefill  # noqa: F401

pytestmark = pytest.mark.gpu

PKV_ERR_TIMEOUT = 10


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 4, 2)])
def test_an_expired_wait_over_pools_with_block_scales(pkv, kind, d, hq, hkv):
    b = Batch(50, kind, [40, 200], [500, 90], hkv, d)
    q, qt = bf16_rows(b.rng, b.T, hq, d)
    out = torch.full((b.T, hq, d), 7.0, device="cuda")
    pkv.test_arm_prefill_stall(1)
    prefill(pkv, b, qt, 0.1, out=out)
    torch.cuda.synchronize()
    status, detail = pkv.get_error()
    assert status == PKV_ERR_TIMEOUT and 0x100 <= detail < 0x112
    assert torch.all(out == 7.0)
    check(b, prefill(pkv, b, qt, 0.1, out=out), q, 0.1)
    assert pkv.get_error()[0] == 0


def test_the_hook_rejects_negative_counts(pkv):
    with pytest.raises(pkv.PKVError):
        pkv.test_arm_prefill_stall(-1)
    pkv.test_arm_prefill_stall(0)


@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 4, 2)])
def test_an_expired_wait_over_bf16_pools(pkv, d, hq, hkv):
    w = W.make_paged("prefill_stall", 24, hq, hkv, d, [540, 290], [40, 200])
    ds = DeviceStep(w)
    pkv.cache_write(ds.k, ds.v, ds.k_new, ds.v_new, ds.slots)
    ws = pkv.new_workspace(pkv.prefill_workspace_size(2, w.num_tokens, hq, hkv, d, w.max_context_len))
    out = torch.full((w.num_tokens, hq, d), 7.0, device="cuda")

    def call():
        pkv.chunked_prefill_attention(ds.k, ds.v, ds.q, ds.qsl, ds.ctx, ds.tables, w.max_context_len, w.scale, out=out,
                                      workspace=ws, query_start_loc_host=w.query_start_loc)
        torch.cuda.synchronize()
        return pkv.get_error()

    pkv.test_arm_prefill_stall(1)
    status, detail = call()
    assert status == PKV_ERR_TIMEOUT and 0x100 <= detail < 0x112
    assert torch.all(out == 7.0)
    assert call()[0] == 0
    _, _, ref = oracle.run_step(w)
    assert_close(out.cpu().numpy(), ref, "prefill after a timeout")
