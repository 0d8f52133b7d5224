"""Rotary positions with frequencies of many turns a position, against the
fp64 oracle: an angle of p f radians is off by 2^-47 of its size, however many
whole turns that is (the tolerance of test_gpu_rotary.py)."""
import numpy as np
import pytest

from gpu_helpers import dev_tensor
from test_gpu_rotary import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("lo,hi", [(1e2, 1e7), (1e7, 1e9), (1e9, 1e11)])
def test_frequencies_of_many_turns(pkv, lo, hi, adjacent):
    b = Batch(700, 9, 2, 2, 64, 64, [32], False, adjacent)
    b.pos[0] = [0, 1, -1, 2, 3, -5, 7, 11, -13]
    b.f = (np.geomspace(lo, hi, 32) * np.where(np.arange(32) % 2, -1, 1)).astype(np.float32)
    q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f), adjacent_pairs=adjacent)
    assert pkv.get_error() == (0, 0)
    b.check_bf16(q, b.q, "q")
    b.check_bf16(k, b.k, "k")


def test_lengths_are_kept_at_any_frequency(pkv):
    """Where the angle says nothing any more, a pair is still only turned:
    its squared length changes by the two bf16 roundings, 2^-8 of a value
    each, so by less than 2^-6."""
    b = Batch(701, 5, 2, 2, 64, 64, [32], False, False)
    b.f = np.geomspace(1e12, 3e38, 32).astype(np.float32)
    q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f))
    for got, x in ((q, b.q), (k, b.k)):
        pair = lambda t: (t.float()[..., :32] ** 2 + t.float()[..., 32:] ** 2).double().cpu().numpy()
        assert np.all(np.abs(pair(got) - pair(x)) <= 2.0 ** -6 * pair(x))
