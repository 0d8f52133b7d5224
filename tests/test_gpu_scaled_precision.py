"""Precision of attention over 8-bit pools with a scale per block and head
where it can be lost: V scales far apart in one context, sums over long
contexts.  Against the float64 oracle; the tolerance is that of
scaled_batch.attention_tolerance unless a test derives its own."""
import numpy as np
import pytest
import torch

from scaled_batch import Batch, bf16_rows
from test_gpu_scaled_attention import KINDS, check, decode, pkv, prefill  # noqa: F401

pytestmark = pytest.mark.gpu

# Powers of the V scales of a context's blocks: the least beside larger ones (a
# block of zeros has the least), steps up and down.
POWERS = [[-100, 40], [40, -100], [-100, 116], [116, -100], [-100, 0, 116], [116, 0, -100], [-60, 90], [0, 116, -100, 50]]


def spread_v_scales(b, powers, stride):
    """Runs of `stride` blocks of each sequence take the V scales 2^power in turn; blocks at the least scale hold
    zeros."""
    for s, n in enumerate(b.lens):
        for i in range(-(-int(n) // 16)):
            power = powers[min(i // stride, len(powers) - 1)]
            b.scales[b.tables[s, i], :, 1] = np.float32(2.0 ** power)
            if power == -100:
                b.v[b.tables[s, i]] = 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("powers", POWERS)
@pytest.mark.parametrize("d,g", [(64, 1), (128, 2), (128, 8)])
def test_v_scales_far_apart_decode(pkv, kind, powers, d, g):
    """Scales that lie far apart within a stage's two blocks, between the stages of a warp, between warps, between the
    parts of a split context: every key counts in the sum of the weights.  (With equal scores 16 zero rows and one
    row v give v / 17.)"""
    for stride, part in ((1, 0), (2, 0), (12, 0), (40, 0), (1, 1), (3, 3), (20, 7)):
        b = Batch(stride + 100 * part, kind, [1] * 3, [16, 16 * 2 * stride + 4, 40 * 16], 2, d)
        spread_v_scales(b, powers, stride)
        for size in (0.0, 1.0):
            q, qt = bf16_rows(b.rng, b.T, 2 * g, d, size=size)
            check(b, decode(pkv, b, qt, d ** -0.5, partition_blocks=part), q, d ** -0.5)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("powers", POWERS)
@pytest.mark.parametrize("d,g", [(64, 1), (128, 2)])
def test_v_scales_far_apart_prefill(pkv, kind, powers, d, g):
    """The same within a tile of 128 keys, and from tile to tile."""
    for stride in (1, 3, 8, 17):
        b = Batch(stride, kind, [17, 150, 1], [0, 16 * 4 * stride, 40], 2, d)
        spread_v_scales(b, powers, stride)
        for size in (0.0, 1.0):
            q, qt = bf16_rows(b.rng, b.T, 2 * g, d, size=size)
            check(b, prefill(pkv, b, qt, d ** -0.5), q, d ** -0.5)
    assert pkv.get_error()[0] == 0
