"""Linear prefill with device lengths that are not the host's: reported, and
nothing is made from memory that the call has not written."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev_tensor
from test_gpu_linear import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


@pytest.mark.parametrize("lens,host,broken", [
    ([64, 192], [0, 128, 256], 1),           # as many chunks, but a border lies inside the second sequence
    ([192, 64], [0, 128, 256], 0),           # inside the first
    ([128, 128], [0, 128, 192], None),       # one chunk more than the host saw, which the last range has room for
    ([128, 192], [0, 128, 192], 1),          # two more: past the last range
])
@pytest.mark.parametrize("past", [0, 5])
def test_a_border_the_plan_did_not_put_inside_a_sequence(pkv, lens, host, broken, past):
    """Two blocks of q heads to a state and ranges of two chunks, none of
    which the host's lengths cut.  The broken sequence's rows are zero where
    they are written and its state is not stored; the other is as usual."""
    hq, hkv, d = 2, 1, 64
    b = Batch(400 + lens[0], lens, [past] * 2, hq, hkv, d)
    ws = torch.full((pkv.linear_prefill_workspace_size(2, b.T, hq, hkv, d),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((b.T, hq, d), 7.0, device="cuda")
    pkv.linear_prefill_attention(*b.args(), dev_tensor(b.qsl), dev_tensor(b.slots), dev_tensor(b.ctx), b.scale,
                                 new_slots=dev_tensor(b.new), out=out, workspace=ws,
                                 query_start_loc_host=np.array(host, np.int32))
    st, detail = pkv.get_error()
    assert st == 9 and detail in (broken, 2)  # 2: the number of chunks is not the host's
    want, after = b.oracle()
    bound, bound_after = b.oracle(absolute=True)
    got = f64(out)
    states = b.states.double().cpu().numpy()
    for s in range(2):
        rows = slice(int(b.qsl[s]), int(b.qsl[s + 1]))
        i = int(b.new[s])
        if s == broken:
            assert np.all((got[rows] == 0) | (got[rows] == 7)) and np.any(got[rows] == 0)
            assert np.array_equal(states[i].astype(np.float32), b.S0[i], equal_nan=True)
        else:
            c = (40 + 4 * lens[s]) * 2.0 ** -24
            assert np.all(np.abs(got[rows] - want[rows]) <= c * bound[rows] + 1e-37)
            assert np.all(np.abs(states[i] - after[i]) <= c * bound_after[i] + 1e-37)
