"""Pins of the linear-attention oracle (no GPU)."""
import numpy as np
import pytest

from oracle import linear as L


def _batch(rng, lens, hq, hkv, d):
    T = sum(lens)
    return (rng.standard_normal((T, hq, d)), rng.standard_normal((T, hkv, d)), rng.standard_normal((T, hkv, d)),
            np.concatenate([[0], np.cumsum(lens)]))


@pytest.mark.parametrize("group", [1, 2])
def test_equals_the_double_sum(group):
    """out_t = scale (lam^(t+1) q S0 + sum_(s<=t) lam^(t-s) (q_t . k_s) v_s)."""
    rng = np.random.default_rng(3)
    hkv, d, n = 2, 4, 7
    q, k, v, qsl = _batch(rng, [n], hkv * group, hkv, d)
    g = np.array([-0.3, -0.01])
    S0 = rng.standard_normal((1, hkv, d, d))
    out, after = L.attend(S0, g, q, k, v, qsl, [0], [n + 5], 0.5)
    for h in range(hkv * group):
        lam = np.exp(g[h // group])
        for t in range(n):
            want = lam ** (t + 1) * q[t, h] @ S0[0, h // group]
            for s in range(t + 1):
                want = want + lam ** (t - s) * (q[t, h] @ k[s, h // group]) * v[s, h // group]
            assert np.allclose(out[t, h], 0.5 * want, rtol=1e-12)
    want = sum(np.exp(g[1]) ** (n - 1 - s) * np.outer(k[s, 1], v[s, 1]) for s in range(n))
    assert np.allclose(after[0, 1], np.exp(g[1]) ** n * S0[0, 1] + want, rtol=1e-12)


def test_first_token_and_no_decay_and_no_memory():
    rng = np.random.default_rng(4)
    q, k, v, qsl = _batch(rng, [3], 1, 1, 4)
    out, _ = L.attend(np.full((1, 1, 4, 4), 9.0), [0.0], q, k, v, qsl, [0], [3], 1.0)
    assert np.allclose(out[0, 0], (q[0, 0] @ k[0, 0]) * v[0, 0])
    assert np.allclose(out[2, 0], sum((q[2, 0] @ k[s, 0]) * v[s, 0] for s in range(3)))
    out, _ = L.attend(np.full((1, 1, 4, 4), 9.0), [-np.inf], q, k, v, qsl, [0], [9], 1.0)
    assert np.allclose(out[2, 0], (q[2, 0] @ k[2, 0]) * v[2, 0])


def test_chunks_equal_one_call_and_slots_are_kept_apart():
    rng = np.random.default_rng(5)
    q, k, v, _ = _batch(rng, [9], 2, 1, 4)
    S = rng.standard_normal((3, 1, 4, 4))
    whole, end = L.attend(S, [-0.2], q, k, v, [0, 9], [1], [9], 1.0, new_slots=[2])
    assert np.array_equal(end[:2], S[:2])
    a, mid = L.attend(S, [-0.2], q[:4], k[:4], v[:4], [0, 4], [1], [4], 1.0)
    b, end2 = L.attend(mid, [-0.2], q[4:], k[4:], v[4:], [0, 5], [1], [9], 1.0)
    assert np.allclose(whole, np.concatenate([a, b]), rtol=1e-12)
    assert np.allclose(end[2], end2[1], rtol=1e-12) and np.array_equal(end2[[0, 2]], S[[0, 2]])


def test_skips():
    rng = np.random.default_rng(6)
    q, k, v, qsl = _batch(rng, [2, 0, 1, 1, 2], 1, 1, 4)
    S = rng.standard_normal((4, 1, 4, 4))
    # a shorter context, no rows, no state to go on from, a fresh sequence that stores nothing, a slot past the pool
    out, after = L.attend(S, [-0.1], q, k, v, qsl, [0, 1, -1, -1, 4], [1, 7, 5, 1, 8], 1.0)
    assert np.all(out[:3] == 0) and np.any(out[3] != 0) and np.all(out[4:] == 0)
    assert np.array_equal(after, S)
