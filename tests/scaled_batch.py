"""Batches over 8-bit pools with a scale per block and head, shared by the GPU tests."""
import numpy as np
import torch

from oracle import scaled as S

NAN_CODE = {np.int8: np.int8(-128), np.uint8: np.uint8(0x7F)}


def bf16_rows(rng, *shape, size=1.0):
    """float32 values of bf16 rows, and their CUDA tensor."""
    x = S.bf16_values(S.to_bf16_bits((size * rng.standard_normal(shape)).astype(np.float32)))
    return x, torch.from_numpy(x).bfloat16().cuda()


def to_dev(pool):
    """An int8 pool as it is, e4m3 codes as float8_e4m3fn."""
    t = torch.from_numpy(pool).cuda()
    return t if pool.dtype == np.int8 else t.view(torch.float8_e4m3fn)


def to_host(t):
    return t.cpu().numpy() if t.dtype == torch.int8 else t.view(torch.uint8).cpu().numpy()


class Batch:
    """Sequences of new[i] rows after past[i] earlier ones over scattered
    blocks.  Rows behind a context, blocks that nobody holds and their scales
    are poisoned (NaN codes, -128 in int8; NaN scales)."""

    def __init__(self, seed, kind, new, past, hkv, d, spread=0.5, size=1.0, empty=False):
        rng = self.rng = np.random.default_rng(seed)
        self.kind, self.new, self.past, self.hkv, self.d = kind, list(new), list(past), hkv, d
        self.lens = np.array([a + b for a, b in zip(new, past)], np.int32)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.start[-1])
        used = [-(-int(n) // 16) for n in self.lens]
        self.nb = sum(used) + 3
        ids = rng.permutation(self.nb).astype(np.int32)
        self.tables = np.full((len(new), max(used + [1])), -7, np.int32)  # entries past a context are never read
        at = 0
        for s, u in enumerate(used):
            self.tables[s, :u] = ids[at:at + u]
            at += u
        self.k = np.full((self.nb, hkv, 16, d), NAN_CODE[kind], kind)
        self.v = self.k.copy()
        self.scales = np.full((self.nb, hkv, 2), np.nan, np.float32)
        top = S.largest(self.k)
        held = self.past if empty else self.lens
        for s in range(len(new)):
            for b in range(-(-int(held[s]) // 16)):
                rows = min(16, int(held[s]) - 16 * b)
                block = self.tables[s, b]
                for pool in (self.k, self.v):
                    x = rng.standard_normal((hkv, rows, d)) * top / 3
                    pool[block, :, :rows] = S.encode(x.astype(np.float32), pool)
                self.scales[block] = size * 3 / top * np.exp(spread * rng.standard_normal((hkv, 2)))

    def dev(self):
        """Device copies: pools, scales, start, lens, tables."""
        return (to_dev(self.k), to_dev(self.v), torch.from_numpy(self.scales).cuda(),
                torch.from_numpy(self.start).cuda(), torch.from_numpy(self.lens).cuda(),
                torch.from_numpy(self.tables).cuda())


def attention_tolerance(exact, context, scales):
    """Bound of |got - out| per element, [T][Hq][d], for exact = what the oracle's attention returns.

    A score is a sum of d exact products in fp32; tensor cores and FMAs lose at
    most 2^-23 of the partial sums at each of d / 16 to d / 4 steps, and the
    factor of scale, block scale and log2 e three roundings: together below
    2^-18 of the sum of the terms' sizes.  A weight is off by the exponential
    of that, by its own exponential (2^-21) and by the log2 of its V scale
    (2^-23 of it, where the kernel adds it to the exponent), and so is the sum
    of weights.  P in two fp16 terms is off by 2^-22; the sums of P V lose up
    to 2^-23 of their size at each 16 keys.  Two fp16 terms and flushed
    exponentials end at 2^-36 of the largest P, which the reference maximum
    may be below by 2^3: each key adds 2^-33 of the largest weight, times its
    V scale, to the sum, times its code.
    """
    out, size, terms, peak = exact
    logs = np.abs(np.log2(np.where(np.isfinite(scales) & (scales > 0), scales, 1.0))).max()
    weight = 2.0 ** -18 * terms[..., None] + 2.0 ** -21 + 2.0 ** -23 * logs
    return (np.expm1(np.minimum(2 * weight, 50.0)) + 2.0 ** -21 + (context / 16 + 8) * 2.0 ** -23) * size + \
        context * 2.0 ** -33 * peak[..., None]
