"""The chunked form of linear attention keeps fp32 values whole in its
tensor-core products: the batches of linear_terms.py, whose tolerances a lost
bf16 term fails (test_linear_terms.py plants one on the CPU), and a join over
many ranges by the norm of the outputs."""
import numpy as np
import pytest
import torch

import linear_terms as T
from gpu_helpers import dev_tensor
from test_gpu_linear import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


def run(pkv, b):
    """Outputs and the state after the call, read from slot 1, stored to 0."""
    rows = b.q.shape[0]
    q, k, v = (torch.from_numpy(np.asarray(x, np.float32)).bfloat16().cuda() for x in (b.q, b.k, b.v))
    states = dev_tensor(np.stack([np.full_like(b.S0, np.nan), b.S0]))
    qsl = np.array([0, rows], np.int32)
    i32 = lambda x: dev_tensor(np.array([x], np.int32))
    out = pkv.linear_prefill_attention(states, dev_tensor(b.g), q, k, v, dev_tensor(qsl), i32(1), i32(rows + b.past),
                                       b.scale, new_slots=i32(0), query_start_loc_host=qsl)
    assert pkv.get_error() == (0, 0)
    return f64(out), states[0].double().cpu().numpy()


# One block; q heads dealt to blocks; rows that end inside a chunk.
SHAPES = [(64, 1, 1, 64), (64, 1, 1, 128), (50, 8, 2, 64), (50, 8, 2, 128), (64, 16, 8, 128), (33, 32, 8, 64)]


@pytest.mark.parametrize("rows,hq,hkv,d", SHAPES)
def test_weighted_scores_are_whole(pkv, rows, hq, hkv, d):
    b = T.Scores(800, rows, hq, hkv, d)
    out, _ = run(pkv, b)
    assert T.worst(out, b.out()) <= b.tol


# ... and chunks in one range and cut into ranges.
@pytest.mark.parametrize("rows,hq,hkv,d", SHAPES + [(300, 16, 8, 128), (300, 4, 2, 64), (1000, 1, 1, 128), (5, 4, 2, 64)])
def test_states_are_whole(pkv, rows, hq, hkv, d):
    b = T.States(801, rows, hq, hkv, d)
    out, after = run(pkv, b)
    assert T.worst(out, b.out()) <= b.tol
    assert np.array_equal(after, b.state())


@pytest.mark.parametrize("rows,hq,hkv,d", SHAPES)
def test_decayed_values_are_whole(pkv, rows, hq, hkv, d):
    b = T.Values(802, rows, hq, hkv, d)
    out, after = run(pkv, b)
    assert np.all(out == 0)
    assert T.worst(after, b.state()) <= b.tol


@pytest.mark.parametrize("rows,hq,hkv,d", [(300, 16, 8, 128), (300, 8, 8, 64), (290, 4, 2, 128), (257, 2, 1, 64)])
def test_decayed_values_of_a_cut_sequence_are_whole(pkv, rows, hq, hkv, d):
    """Five chunks in five ranges at most: three joins between the first
    range, which holds the values, and the last."""
    b = T.Values(803, rows, hq, hkv, d, joins=3)
    out, after = run(pkv, b)
    assert np.all(out == 0)
    assert T.worst(after, b.state()) <= b.tol


def test_a_join_of_many_ranges_by_the_norm(pkv):
    """100,000 tokens of one head of 64 that forgets 2e-4 a token, so that a
    state lasts 1 / (1 - exp(-0.0128)) = 79 chunks.  A truncating sum loses
    less than 2^-23 of what it has: four a chunk in the update and one in the
    two roundings of the decay, over 79 chunks; 16 in an output's own products,
    sums and factors; four at each of the 10 joins a state lasts."""
    b = Batch(72, [100000], [4], 1, 1, 64)
    b.g[:] = -2e-4
    out = f64(b.prefill(pkv))
    assert pkv.get_error() == (0, 0)
    want, after = b.oracle()
    tol = (5 * 79 + 16 + 4 * 10) * 2.0 ** -23
    for at in range(0, b.T, 64):
        rows = slice(at, at + 64)
        assert np.linalg.norm(out[rows] - want[rows]) <= tol * np.linalg.norm(want[rows]), at
    i = int(b.new[0])
    state = b.states[i].double().cpu().numpy()
    assert np.linalg.norm(state - after[i]) <= tol * np.linalg.norm(after[i])


@pytest.mark.parametrize("lens,past,hq,hkv,d", [
    ([300], [0], 16, 8, 128), ([300], [6], 4, 2, 64), ([64, 130, 200], [5, 0, 3], 8, 2, 128),
    ([64] * 8, [4] * 8, 8, 8, 64), ([320, 1, 70, 2], [9, 9, 0, 4], 8, 4, 128)])
def test_errors_are_those_of_fp32_sums(pkv, lens, past, hq, hkv, d):
    """At most five chunks to a sequence, every head and state by its norm, to
    1e-6.  A truncating sum loses half a step on average, 0.72 2^-24 of a
    value, all the same way.  Scores and P V are 8 + 4 such sums at head_dim
    128, the partial ones two thirds of the whole on average: 3.4e-7.  Four
    chunks' updates, four sums each, two thirds: 4.6e-7, and 8 in the outputs'
    product with the state: 2.3e-7; together less than 7e-7 of a norm, and the
    roundings to nearest, which are independent, 1e-7."""
    b = Batch(804 + len(lens), lens, past, hq, hkv, d)
    out = f64(b.prefill(pkv))
    assert pkv.get_error() == (0, 0)
    want, after = b.oracle()
    states = b.states.double().cpu().numpy()
    for s in range(len(lens)):
        rows = slice(int(b.qsl[s]), int(b.qsl[s + 1]))
        for h in range(hq):
            err = np.linalg.norm(out[rows, h] - want[rows, h])
            assert err <= 1e-6 * np.linalg.norm(want[rows, h]), (s, h, err / np.linalg.norm(want[rows, h]))
        i = int(b.new[s])
        for h in range(hkv):
            assert np.linalg.norm(states[i, h] - after[i, h]) <= 1e-6 * np.linalg.norm(after[i, h]), (s, h)
