"""Oracle of 8-bit pools with a scale for each (block, kv head) -- TEST INFRASTRUCTURE ONLY.

Only the tests and ``__graft_entry__.smoke()`` may import this module.  It
shares no code with the CUDA library.

Pools are uint8 (e4m3 codes) or int8 arrays [num_blocks][Hkv][16][d], scales
float32 [num_blocks][Hkv][2] (K, V).  Everything goes row by row and block by
block, in the order of the definition:

- append: per touched (block, head), scale = max(old, amax * (1 / L), 2^-100)
  and code(x) = nearest(x * (1 / scale)), each operation rounded to float32;
  old is 0 for a block whose first row is new, and its earlier rows are
  encoded again from value(code) * (old * (1 / scale)) where the scale grew;
- read: value(code) * scale in float32, rounded to bf16;
- attention: float64 over value(code) * scale.

Parity status: pinned by ``tests/test_oracle_scaled.py``.
"""
from __future__ import annotations

import numpy as np

from . import fp8

LEAST, MOST = np.float32(2.0 ** -100), np.float32(2.0 ** 122)


def largest(pool) -> float:
    return 127.0 if pool.dtype == np.int8 else 448.0


def values(codes) -> np.ndarray:
    """float64 values of codes."""
    return codes.astype(np.float64) if codes.dtype == np.int8 else fp8.value(codes)


def encode(x, like) -> np.ndarray:
    """Nearest codes of float32 x, ties to even, saturating; NaN is 0 in int8."""
    if like.dtype == np.int8:
        y = np.where(np.isnan(x), 0.0, np.clip(x.astype(np.float64), -127.0, 127.0))
        return np.rint(y).astype(np.int8)
    return fp8.encode(x)


def used_scale(s) -> np.float32:
    return np.float32(s) if LEAST <= s <= MOST else LEAST


def bf16_values(bits) -> np.ndarray:
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def to_bf16_bits(x) -> np.ndarray:
    """float32 -> bf16 bits, to nearest even (finite values)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _rows(start, context_lens, tables, num_blocks, num_tokens, wide):
    """(sequence, block id, rows of the block, first token) of a batch, in order; bad sequences and ids are left out."""
    for s in range(len(context_lens)):
        a, b, n = int(start[s]), int(start[s + 1]), int(context_lens[s])
        if a < 0 or b <= a or b > num_tokens or n < b - a or n > wide * 16:
            continue
        at = n - (b - a)
        while at < n:
            r, block = at % 16, int(tables[s][at // 16])
            count = min(16 - r, n - at)
            if 0 <= block < num_blocks:
                yield s, block, range(r, r + count), a + at - (n - (b - a))
            at += count


def append(k_pool, v_pool, scales, k_new, v_new, start, context_lens, tables):
    """In place; k_new/v_new float32 values [T][Hkv][d] of bf16 rows."""
    nb, hkv = k_pool.shape[:2]
    with np.errstate(invalid="ignore", over="ignore"):
        for _, block, rows, t in _rows(start, context_lens, tables, nb, len(k_new), np.shape(tables)[1]):
            for which, (pool, new) in enumerate(((k_pool, k_new), (v_pool, v_new))):
                inv_l = np.float32(1.0 / largest(pool))
                for h in range(hkv):
                    x = np.asarray(new[t:t + len(rows), h], dtype=np.float32)
                    amax = np.max(np.abs(x[np.isfinite(x)]), initial=np.float32(0))
                    old = used_scale(scales[block, h, which]) if rows[0] > 0 else np.float32(0)
                    scale = max(old, np.float32(amax * inv_l), LEAST)
                    inv = np.float32(np.float32(1) / scale)
                    if rows[0] > 0 and scale > old:
                        ratio = np.float32(old * inv)
                        held = values(pool[block, h, :rows[0]]).astype(np.float32)
                        pool[block, h, :rows[0]] = encode(held * ratio, pool)
                    pool[block, h, rows[0]:rows[-1] + 1] = encode(x * inv, pool)
                    scales[block, h, which] = scale


def read(k_pool, v_pool, scales, start, context_lens, tables, num_tokens):
    """float32 values (before the rounding to bf16) [T][Hkv][d] of K and V; rows nobody owns are NaN."""
    nb, hkv, _, d = k_pool.shape
    out = [np.full((num_tokens, hkv, d), np.nan, dtype=np.float32) for _ in range(2)]
    for _, block, rows, t in _rows(start, context_lens, tables, nb, num_tokens, np.shape(tables)[1]):
        for which, pool in enumerate((k_pool, v_pool)):
            for h in range(hkv):
                x = values(pool[block, h, rows[0]:rows[-1] + 1]).astype(np.float32)
                out[which][t:t + len(rows), h] = x * used_scale(scales[block, h, which])
    return out


def attention(k_pool, v_pool, scales, q, start, context_lens, tables, scale):
    """float64 causal attention of the rows at the ends of the contexts, out [T][Hq][d], and what its error goes by:
    the weighted sum of |v| [T][Hq][d], the largest sum of |q k| [T][Hq], the largest weight times V scale times
    largest code [T][Hq].  An empty context gives zero rows."""
    q = np.asarray(q, dtype=np.float64)
    T, hq, d = q.shape
    hkv = k_pool.shape[1]
    out, size, terms, peak = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq)), np.zeros((T, hq))
    for s in range(len(context_lens)):
        a, b, n = int(start[s]), int(start[s + 1]), int(context_lens[s])
        if b <= a or n == 0:
            continue
        pos = np.arange(n)
        blocks = np.asarray(tables[s])[pos // 16]
        sc = np.where((scales >= LEAST) & (scales <= MOST), scales, LEAST).astype(np.float64)[blocks]
        K = values(k_pool[blocks, :, pos % 16]) * sc[..., 0, None]
        V = values(v_pool[blocks, :, pos % 16]) * sc[..., 1, None]
        for h in range(hq):
            g = h // (hq // hkv)
            for t in range(a, b):
                m = n - b + t + 1
                x = scale * (K[:m, g] @ q[t, h])
                w = np.exp(x - x.max())
                w /= w.sum()
                out[t, h], size[t, h] = w @ V[:m, g], w @ np.abs(V[:m, g])
                terms[t, h] = abs(scale) * np.max(np.abs(K[:m, g]) @ np.abs(q[t, h]))
                peak[t, h] = np.max(w * sc[:m, g, 1]) * largest(v_pool)
    return out, size, terms, peak
