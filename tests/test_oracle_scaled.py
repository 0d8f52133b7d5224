"""Pins of the oracle of 8-bit pools with a scale per block and head (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import fp8
from oracle import scaled as S

KINDS = [np.int8, np.uint8]


def pools(kind, nb=4, hkv=2, d=8):
    return (np.zeros((nb, hkv, 16, d), kind), np.zeros((nb, hkv, 16, d), kind),
            np.full((nb, hkv, 2), np.nan, np.float32))


def rows(rng, t, hkv=2, d=8, size=1.0):
    x = (size * rng.standard_normal((t, hkv, d))).astype(np.float32)
    return S.bf16_values(S.to_bf16_bits(x))


@pytest.mark.parametrize("kind", KINDS)
def test_a_full_block_is_within_half_a_step(kind):
    rng = np.random.default_rng(1)
    k, v, sc = pools(kind)
    kn, vn = rows(rng, 16), rows(rng, 16, size=100.0)
    S.append(k, v, sc, kn, vn, [0, 16], [16], [[2]])
    for which, (pool, x) in enumerate(((k, kn), (v, vn))):
        for h in range(2):
            s = sc[2, h, which]
            amax = np.abs(x[:, h]).max()
            assert s == np.float32(amax * np.float32(1 / S.largest(pool)))
            got = S.values(pool[2, h]) * float(s)
            step = np.full(got.shape, float(s)) if kind == np.int8 else np.maximum(np.abs(x[:, h]) / 8, s * 2.0 ** -9)
            assert np.all(np.abs(got - x[:, h]) <= 0.5 * step * (1 + 2 ** -20))
            assert np.abs(S.values(pool[2, h])).max() == S.largest(pool)
    assert np.isnan(sc[[0, 1, 3]]).all() and not k[[0, 1, 3]].any()


@pytest.mark.parametrize("kind", KINDS)
def test_the_scale_grows_and_never_shrinks(kind):
    k, v, sc = pools(kind, hkv=1, d=1)
    one = np.ones((1, 1, 1), np.float32)
    S.append(k, v, sc, one, one, [0, 1], [1], [[0]])
    assert sc[0, 0, 0] == np.float32(1 / S.largest(k)) and S.values(k[0, 0, 0])[0] == S.largest(k)
    S.append(k, v, sc, 4 * one, one, [0, 1], [2], [[0]])          # K grows fourfold, V stays
    assert sc[0, 0, 0] == np.float32(4 * np.float32(1 / S.largest(k))) and sc[0, 0, 1] == np.float32(1 / S.largest(k))
    assert S.values(k[0, 0, :2])[:, 0].tolist() == ([32.0, 127.0] if kind == np.int8 else [112.0, 448.0])
    assert S.values(v[0, 0, :2])[:, 0].tolist() == [S.largest(k)] * 2
    S.append(k, v, sc, 0 * one, one, [0, 1], [3], [[0]])
    assert sc[0, 0, 0] == np.float32(4 * np.float32(1 / S.largest(k)))
    S.append(k, v, sc, one, one, [0, 1], [1], [[0]])              # the block starts anew
    assert sc[0, 0, 0] == np.float32(1 / S.largest(k))


@pytest.mark.parametrize("kind", KINDS)
def test_zero_rows_infinities_and_nan(kind):
    k, v, sc = pools(kind, hkv=1, d=4)
    x = np.array([[[0, 0, 0, 0]], [[np.inf, -np.inf, 2, np.nan]]], np.float32)
    S.append(k, v, sc, x[:1], x[1:], [0, 1], [1], [[3]])
    assert sc[3, 0, 0] == np.float32(2.0 ** -100) and not k[3, 0, 0].any()
    top = S.largest(v)
    got = S.values(v[3, 0, 0])
    assert got[:3].tolist() == [top, -top, top] and (got[3] == 0 if kind == np.int8 else np.isnan(got[3]))


def test_codes_agree_with_torch():
    """int8 against torch's rounding (to even), e4m3 against its conversion."""
    x = np.concatenate([np.arange(-130, 130, 0.25), [0.5, 1.5, 2.5, -0.5]]).astype(np.float32)
    want = torch.from_numpy(x).round().clamp(-127, 127).to(torch.int8).numpy()
    assert np.array_equal(S.encode(x, np.zeros(1, np.int8)), want)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.value(S.encode(x, np.zeros(1, np.uint8))), fp8.value(want))


@pytest.mark.parametrize("kind", KINDS)
def test_splitting_the_rows_over_calls(kind):
    """Codes that carry their block's largest value from the start do not depend on the calls' borders."""
    rng = np.random.default_rng(2)
    x = rows(rng, 40)
    x[::16] = 8.0  # the largest value is in each block's first row
    tables = [[1, 3, 0]]
    a, b = pools(kind), pools(kind)
    S.append(*a, x, -x, [0, 40], [40], tables)
    at = 0
    for n in (5, 11, 1, 20, 3):
        S.append(*b, x[at:at + n], -x[at:at + n], [0, n], [at + n], tables)
        at += n
    assert all(np.array_equal(p, q, equal_nan=p.dtype == np.float32) for p, q in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
def test_read_is_the_inverse_and_attention_equals_the_plain_sum(kind):
    rng = np.random.default_rng(3)
    p = pools(kind)
    x, y = rows(rng, 23), rows(rng, 23)
    S.append(*p, x, y, [0, 23], [23], [[2, 0]])
    rk, rv = S.read(*p, [0, 23], [23], [[2, 0]], 23)
    step = 1 / 127 if kind == np.int8 else 1 / 16
    assert np.abs(rk - x).max() <= step * np.abs(x).max() and np.abs(rv - y).max() <= step * np.abs(y).max()
    q = rows(rng, 3, hkv=4)
    out, size, terms, _ = S.attention(*p, q, [0, 3], [23], [[2, 0]], 0.5)
    for t in range(3):
        for h in range(4):
            m = 21 + t
            w = np.exp(0.5 * rk[:m, h // 2].astype(float) @ q[t, h].astype(float))
            want = w @ rv[:m, h // 2].astype(float) / w.sum()
            # The read rounds each product to fp32, 2^-24 of it: a score moves by 2^-24 of its terms, a weight by
            # twice that (its own exponential and the sum's), and each V by 2^-24.
            assert np.all(np.abs(out[t, h] - want) <= (2 * terms[t, h] + 1.01) * 2.0 ** -24 * size[t, h])


def test_bad_sequences_store_nothing():
    k, v, sc = pools(np.int8)
    x = rows(np.random.default_rng(4), 6)
    S.append(k, v, sc, x, x, [0, 2, 4, 6], [1, 40, 4], [[0, 1], [2, 3], [-1, 9]])
    assert np.isnan(sc).all() and not k.any() and not v.any()


# Mistakes in a copy of the oracle's rules that the pins above have to see.
MISTAKES = [
    ("scale = max(old, np.float32(amax * inv_l), LEAST)", "scale = max(np.float32(amax * inv_l), LEAST)"),
    ("ratio = np.float32(old * inv)", "ratio = np.float32(scale * np.float32(1 / old))"),
    ("if rows[0] > 0 else np.float32(0)", "if True else np.float32(0)"),
    ("np.rint(y)", "np.trunc(y)"),
    ("x[np.isfinite(x)]", "np.nan_to_num(x)"),
    ("sc[..., 1, None]", "sc[..., 0, None]"),
    ("m = n - b + t + 1", "m = n"),
    ("(k_pool, k_new), (v_pool, v_new)", "(k_pool, k_new), (v_pool, k_new)"),
]


@pytest.mark.parametrize("right,wrong", MISTAKES)
def test_planted_mistakes_are_seen(right, wrong, monkeypatch):
    import types
    text = open(S.__file__).read()
    assert text.count(right) == 1
    bad = types.ModuleType("oracle.scaled_mistake")
    bad.__package__, bad.__file__ = "oracle", S.__file__
    exec(compile(text.replace(right, wrong), "mistake", "exec"), bad.__dict__)
    for name in ("append", "read", "attention", "values", "encode"):
        monkeypatch.setattr(S, name, getattr(bad, name))
    with pytest.raises((AssertionError, ValueError)):
        for kind in KINDS:
            test_a_full_block_is_within_half_a_step(kind)
            test_the_scale_grows_and_never_shrinks(kind)
            test_zero_rows_infinities_and_nan(kind)
            test_splitting_the_rows_over_calls(kind)
            test_read_is_the_inverse_and_attention_equals_the_plain_sum(kind)
        test_codes_agree_with_torch()
