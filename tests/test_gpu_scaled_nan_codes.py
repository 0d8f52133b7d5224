"""Prefill tiles with a NaN code in V, whose rows are computed again on CUDA
cores: both head dims, CTAs of one q head and of two, tiles split by head,
contexts of several key tiles.  The NaN is where it belongs, every other
element is the oracle's."""
import numpy as np
import pytest

from oracle import scaled as S
from scaled_batch import NAN_CODE, Batch, attention_tolerance, bf16_rows
from test_gpu_scaled_attention import pkv, prefill  # noqa: F401

pytestmark = pytest.mark.gpu

CODE = NAN_CODE[np.uint8]


def check_with_nans(b, got, q, scale):
    exact = S.attention(b.k, b.v, b.scales, q, b.start, b.lens, b.tables, scale)
    held = np.concatenate([b.tables[s, :-(-int(n) // 16)] for s, n in enumerate(b.lens)]).astype(int)
    tol = attention_tolerance(exact, int(b.lens.max()), b.scales[held])
    got = got.double().cpu().numpy()
    nan = np.isnan(exact[0])
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(got), nan)
    assert np.all((np.abs(got - exact[0]) <= tol) | nan)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,hkv", [(1, 2), (2, 2), (8, 1)])
@pytest.mark.parametrize("new,past,place", [
    ([20, 30], [30, 10], 35),           # one key tile
    ([300, 50], [500, 3], 0),           # the first key of several tiles, seen by every row
    ([300, 50], [500, 3], 511),         # the last key of a tile
    ([300, 50], [500, 3], 700),         # in the chunk itself: rows before it do not see it
    ([130, 1, 1], [127, 300, 300], 256),  # the last key of a tile of two rows; a decode row of another sequence
])
def test_a_nan_code_in_v(pkv, d, g, hkv, new, past, place):
    b = Batch(place + d + g, np.uint8, new, past, hkv, d)
    b.v[b.tables[0, place // 16], hkv - 1, place % 16, d - 3] = CODE
    q, qt = bf16_rows(b.rng, b.T, g * hkv, d)
    check_with_nans(b, prefill(pkv, b, qt, d ** -0.5), q, d ** -0.5)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_nan_codes_in_many_tiles(pkv, d):
    """Grids of several waves (no tiles split) with NaN codes in every sequence, at scales far apart."""
    b = Batch(70 + d, np.uint8, [260] * 40, [40] * 40, 2, d)
    for s in range(40):
        b.v[b.tables[s, s % 18], s % 2, s % 16, s] = CODE
        b.scales[b.tables[s, 3], :, 1] = 2.0 ** -100
        b.scales[b.tables[s, 5], :, 1] = 2.0 ** 30
    q, qt = bf16_rows(b.rng, b.T, 4, d)
    check_with_nans(b, prefill(pkv, b, qt, d ** -0.5), q, d ** -0.5)
    assert pkv.get_error()[0] == 0
