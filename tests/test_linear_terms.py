"""The batches of linear_terms.py: they are what the oracle says, and a bf16
term left out of P, S or V~ fails their tolerance (planted here, on the CPU)."""
import numpy as np
import pytest

import linear_terms as T
from oracle import linear as L

CASES = [(T.Scores, 64, 4, 2, 64, {}), (T.Scores, 50, 2, 1, 128, {}), (T.States, 70, 4, 2, 64, {}),
         (T.States, 64, 2, 1, 128, {}), (T.Values, 64, 2, 1, 64, {}), (T.Values, 300, 4, 2, 128, dict(joins=3)),
         (T.Values, 40, 1, 1, 128, {})]


@pytest.mark.parametrize("kind,rows,hq,hkv,d,kw", CASES)
def test_batches_are_what_the_oracle_says(kind, rows, hq, hkv, d, kw):
    b = kind(1, rows, hq, hkv, d, **kw)
    for x in (b.q, b.k, b.v):
        assert np.array_equal(T.to_bf16(x), x)  # exact in bf16
    out, after = L.attend(b.S0[None], b.g, b.q, b.k, b.v, [0, rows], [0], [rows + b.past], b.scale)
    assert np.allclose(out, b.out(), rtol=1e-12, atol=0)
    if b.state() is not None:
        assert np.allclose(after[0], b.state(), rtol=1e-12, atol=0)


@pytest.mark.parametrize("kind,rows,hq,hkv,d,kw", CASES)
def test_a_lost_term_fails(kind, rows, hq, hkv, d, kw):
    b = kind(2, rows, hq, hkv, d, **kw)
    whole, cut = b.out(3), b.out(2)
    if kind is T.Values:
        whole, cut = b.state(3), b.state(2)
    assert T.worst(T.split(whole.astype(np.float32), 3), whole) <= 2 * T.STEP
    assert T.worst(cut, whole) > 1.5 * b.tol
    assert np.mean(np.abs(cut - whole) > b.tol * np.abs(whole)) > 0.02


def test_three_terms_hold_24_bits():
    x = np.random.default_rng(3).standard_normal(10000).astype(np.float32)
    assert np.array_equal(T.split(x, 3), x.astype(np.float64))
    assert not np.array_equal(T.split(x, 2), x.astype(np.float64))
