"""Device row starts that differ from the host's, which the launch is planned
from: what they give rows that no launch takes is reported, the rows that are
taken are right by the device's starts, nothing else is written."""
import numpy as np
import pytest
import torch

from oracle import scaled as S
from scaled_batch import Batch, bf16_rows

pytestmark = pytest.mark.gpu

PKV_ERR_RANGE = 9


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    p.get_error()
    return p


# Host starts, device starts, sequence reported (None: every row has a launch), sequences that are right.
CASES = [
    ([0, 1, 31, 32], [0, 3, 31, 32], 1, [0, 2]),      # two prefill sequences in place of one, one row tile planned
    ([0, 2, 4], [0, 1, 4], 0, [1]),                   # a decode row in a call without a decode launch
    ([0, 1, 2], [0, 2, 2], 0, []),                    # prefill rows in a call without a prefill launch
    ([0, 128, 256], [0, 129, 256], 1, [0]),           # three row tiles where two are planned
    ([0, 40, 80], [0, 60, 80], None, [0, 1]),         # a border moved within the plan
    ([0, 40, 80, 81], [0, 80, 80, 81], None, [0, 2]),  # a sequence that has no rows any more
    ([0, 20, 40, 60], [0, 40, 20, 60], 1, []),        # a start below the one before
]


@pytest.mark.parametrize("pool", ["bf16", "int8"])
@pytest.mark.parametrize("host,device,bad,right", CASES)
def test_starts_that_differ(pkv, pool, host, device, bad, right):
    seqs = len(host) - 1
    past = [300] * seqs
    b = Batch(60, np.int8, [1] * seqs, past, 2, 64)
    b.lens = np.array([301 + 17 * s for s in range(seqs)], np.int32)  # keys past 301 are zeros of block 0
    wide = -(-int(b.lens.max()) // 16)
    tables = np.zeros((seqs, wide), np.int32)
    tables[:, :b.tables.shape[1]] = b.tables
    b.k[tables], b.v[tables] = np.clip(b.k[tables], -127, 127), np.clip(b.v[tables], -127, 127)
    b.scales[~np.isfinite(b.scales)] = 1.0
    T = host[-1]
    q, qt = bf16_rows(b.rng, T, 4, 64)
    out = torch.full((T + 4, 4, 64), 5.0, device="cuda")
    start_host = torch.tensor(host, dtype=torch.int32)
    args = [qt, torch.tensor(device, dtype=torch.int32, device="cuda"), torch.from_numpy(b.lens).cuda(),
            torch.from_numpy(tables).cuda(), int(b.lens.max()), 0.125]
    scales = b.scales.copy()
    if pool == "int8":
        pools = [torch.from_numpy(b.k).cuda(), torch.from_numpy(b.v).cuda()]
        kw = dict(block_scales=torch.from_numpy(scales).cuda())
    else:  # the same codes as bf16 values of 1/16
        scales[:] = 1 / 16
        pools = [(torch.from_numpy(x).cuda().float() / 16).bfloat16() for x in (b.k, b.v)]
        kw = {}
    pkv.chunked_prefill_attention(*pools, *args, out=out[:T], query_start_loc_host=start_host, **kw)
    torch.cuda.synchronize()
    status, detail = pkv.get_error()
    assert (status, detail) == ((0, 0) if bad is None else (PKV_ERR_RANGE, bad))
    got = out.cpu().numpy()
    assert np.all(got[T:] == 5.0)
    for s in right:
        rows = slice(device[s], device[s + 1])
        exact = S.attention(b.k, b.v, scales, q[rows], [0, device[s + 1] - device[s]], b.lens[s:s + 1], tables[s:s + 1],
                            0.125)[0]
        assert np.abs(got[rows] - exact).max() < 2e-3 * max(1.0, np.abs(exact).max())
