"""Precision of attention over 8-bit pools with a scale per block and head
where it can be lost: V scales far apart in one context, sums over long
contexts.  Against the float64 oracle; the tolerance is that of
scaled_batch.attention_tolerance unless a test derives its own."""
import numpy as np
import pytest
import torch

from oracle import scaled as S
from scaled_batch import Batch, bf16_rows, to_dev
from test_gpu_scaled_attention import KINDS, check, decode, pkv, prefill  # noqa: F401

pytestmark = pytest.mark.gpu

# Powers of the V scales of a context's blocks: the least beside larger ones (a
# block of zeros has the least), steps up and down.
POWERS = [[-100, 40], [40, -100], [-100, 116], [116, -100], [-100, 0, 116], [116, 0, -100], [-60, 90],
          [0, 116, -100, 50], [116, 110], [99, 103, 101], [-100, 3], [-100, 4], [-100, 5], [5, -100], [-100, 4, 9]]


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
        for size in (0.0, 8.0):
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
        for size in (0.0, 8.0):
            q, qt = bf16_rows(b.rng, b.T, 2 * g, d, size=size)
            check(b, prefill(pkv, b, qt, d ** -0.5), q, d ** -0.5)
    assert pkv.get_error()[0] == 0


def long_run_of_zeros(kind, zeros, d, rows):
    """A context of `zeros` keys with zero V at the least scale, then one block of scale 1, as a table over four
    blocks.  The first 128 keys have score 0, the other zero rows 2, the last block's keys 0.  Returns the pools, the
    table, q and the float64 out of the last `rows` rows."""
    rng = np.random.default_rng(zeros)
    k, v = np.zeros((4, 1, 16, d), kind), np.zeros((4, 1, 16, d), kind)
    code = np.uint8(0x38) if kind == np.uint8 else np.int8(1)  # 1
    k[1, 0, :, 0] = code
    x = rng.standard_normal((16, d)).astype(np.float32) * 30
    v[2, 0] = S.encode(x, v)
    scales = np.ones((4, 1, 2), np.float32)
    scales[:2, 0, 1] = 2.0 ** -100
    table = np.full(zeros // 16 + 1, 1, np.int32)
    table[:8], table[-1] = 0, 2
    q = np.zeros((rows, 1, d), np.float32)
    q[:, 0, 0] = 2.0
    values = S.values(v[2, 0])
    want = [values[:n].sum(0) / (128 + n + (zeros - 128) * np.exp(2.0)) for n in range(17 - rows, 17)]
    dev = [to_dev(k), to_dev(v), torch.from_numpy(scales).cuda(), torch.from_numpy(table[None]).cuda(),
           torch.tensor([zeros + 16], dtype=torch.int32, device="cuda"), torch.from_numpy(q).bfloat16().cuda()]
    return dev, np.stack(want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_long_run_of_the_least_scale(pkv, kind, d):
    """Sums of 2^(s - log2 vs) over long runs of zero rows stay in fp32.

    A thread sums at most an eighth of the terms one by one, each addition off by 2^-24 of the sum; the other roundings
    are the usual ones, below 2^-18."""
    for zeros in (2 ** 12, 2 ** 17, 2 ** 18, 2 ** 20):
        (k, v, sc, tables, lens, q), want = long_run_of_zeros(kind, zeros, d, 2)
        tol = (zeros / 8 * 2.0 ** -24 + 2.0 ** -18) * np.abs(want)
        start = torch.tensor([0, 2], dtype=torch.int32)
        got = pkv.chunked_prefill_attention(k, v, q, start.cuda(), lens, tables, zeros + 16, 1.0,
                                            query_start_loc_host=start, block_scales=sc)
        assert np.all(np.abs(got[:, 0].double().cpu().numpy() - want) <= tol)
        for part in (0, zeros // 16 + 1):
            got = pkv.decode_attention(k, v, q[1:], tables, lens, zeros + 16, 1.0, block_scales=sc, partition_blocks=part)
            assert np.all(np.abs(got[:, 0].double().cpu().numpy() - want[1:]) <= tol[1:])
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,g", [(64, 1), (64, 8), (128, 1), (128, 2), (128, 4), (128, 8)])
@pytest.mark.parametrize("n", [131072, 100003])
def test_long_contexts_in_one_piece(pkv, kind, d, g, n):
    """Rows of long contexts that one CTA reads do not come out short: V of one sign, all weights equal.

    Of the sum of |w v|: a warp (8 or 12 of them) adds up 64 MMAs, each off by 2^-23, before it adds them to the rest,
    n / 4,096 additions off by 2^-24; the weights' sum goes the same way with 36 additions at a time; P's two terms,
    scales, merge and quotient together are below 2^-20."""
    rng = np.random.default_rng(n + d + g)
    k, v = (np.zeros((600, 1, 16, d), kind) for _ in range(2))
    k[:] = S.encode(rng.standard_normal(k.shape).astype(np.float32) * 30, k)
    v[:] = S.encode(np.abs(rng.standard_normal(v.shape)).astype(np.float32) * 30 + 20, v)
    scales = (0.01 * np.exp(0.1 * rng.standard_normal((600, 1, 2)))).astype(np.float32)
    table = rng.integers(0, 600, -(-n // 16)).astype(np.int32)
    rows = S.values(v) * scales[..., 1, None, None].astype(np.float64)
    want = rows[table, 0].reshape(-1, d)[:n].mean(0)
    q = torch.zeros((1, g, d), dtype=torch.bfloat16, device="cuda")
    tables, lens = torch.from_numpy(table[None]).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda")
    for part in (0, len(table)):
        got = pkv.decode_attention(to_dev(k), to_dev(v), q, tables, lens, n, 0.1, partition_blocks=part,
                                   block_scales=torch.from_numpy(scales).cuda())
        off = np.abs(got[0].double().cpu().numpy() / want - 1).max()
        assert off <= 64 * 2.0 ** -23 + 2 * n / 4096 * 2.0 ** -24 + 36 * 2.0 ** -24 + 2.0 ** -20, f"{off:.2e}"
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,g", [(64, 2), (128, 1), (128, 8)])
@pytest.mark.parametrize("powers", [[-6], [-100, 40], [40, -100, 0], [-6, 1, 8]])
def test_long_items_in_turn(pkv, kind, d, g, powers):
    """One CTA reads long and short contexts one after the other, each warp's state joining its slot several times,
    with V scales and a running maximum that move meanwhile."""
    lens = [20001, 300, 9000, 0, 16]
    b = Batch(80 + g, kind, [1] * 5, [max(n - 1, 0) for n in lens], 2, d)
    b.lens = np.array(lens, np.int32)
    spread_v_scales(b, powers, 300)
    for s, n in enumerate(lens):
        for i in range(0, -(-n // 16), 97):  # K grows along the context
            b.scales[b.tables[s, i], :, 0] *= 1 + i / 300
    q, qt = bf16_rows(b.rng, b.T, 2 * g, d)
    k, v, sc, _, lens_dev, tables = b.dev()
    for part in (0, 4000):
        got = pkv.decode_attention(k, v, qt, tables, lens_dev, max(lens), d ** -0.5, block_scales=sc,
                                   partition_blocks=part)
        check(b, got, q, d ** -0.5)
    assert pkv.get_error()[0] == 0
