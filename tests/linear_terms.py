"""Batches for linear attention whose outputs and states show single fp32
values, so that they tell whether a value went into a matrix product whole.

The chunked form takes its fp32 operands (the weighted scores P, the state S,
the decayed values V~) apart into bf16 terms.  Three terms hold 24 bits;
without the third an element is off by up to 2^-19 of its binade, 1.9e-6, and
5e-7 in the root mean square, which sums over many tokens do not show.  Here
every sum has one element in it.

Tolerances count the roundings an element passes: 2^-24 for a product or a
sum, twice that for a sum of the tensor cores, which may truncate, and for an
exponential of an argument near 0 (two units of a value below 1).
"""
import numpy as np

STEP = 2.0 ** -24


def to_bf16(x):
    """fp32 rounded to bf16, to nearest even, as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def split(x, terms):
    """fp32 in that many bf16 terms, summed again (in 64 bits)."""
    left, out = np.array(x, np.float32), np.zeros(np.shape(x))
    for _ in range(terms):
        t = to_bf16(left)
        out += t
        left = (left - t).astype(np.float32)
    return out


class Scores:
    """One chunk from a zero state, no decay, scale 1.  Every key is 1 in three
    dims and q holds 8 bits of a 24-bit number in each of them, so all scores of
    a row are that number; v of token s is 1 in dim s, so out[t][s] is P[s][t]
    (0 past t).  Two sums at most: the score's, and the three terms'."""
    tol = 4 * STEP

    def __init__(self, seed, rows, hq, hkv, d):
        rng = np.random.default_rng(seed)
        self.g = np.zeros(hkv, np.float32)
        self.scale = 1.0
        self.past = 0
        q, self.k, self.v = np.zeros((rows, hq, d)), np.zeros((rows, hkv, d)), np.zeros((rows, hkv, d))
        part = rng.integers(0, 256, (rows, hq, 3))
        part[:, :, 0] |= 128
        q[:, :, :3] = part * np.array([1.0, 2.0 ** -8, 2.0 ** -16])
        self.q = q
        self.k[:, :, :3] = 1
        self.v[np.arange(rows), :, np.arange(rows)] = 1
        self.S0 = np.zeros((hkv, d, d), np.float32)

    def out(self, terms=3):
        rows, hq, d = self.q.shape
        P = split(self.q.sum(-1), terms)                      # [t][h]
        seen = np.arange(d)[None, :] <= np.arange(rows)[:, None]
        seen[:, rows:] = False
        return P[:, :, None] * seen[:, None, :]

    def state(self, terms=3):
        return None


class States:
    """Rows that go on from a state of full fp32 values without decay; q of
    row t is 1 in one dim, k and v are 0: out[t] is a row of the state, the sum
    of its three terms, and the state stays to the bit."""
    tol = 4 * STEP

    def __init__(self, seed, rows, hq, hkv, d):
        rng = np.random.default_rng(seed)
        self.g = np.zeros(hkv, np.float32)
        self.scale = 1.0
        self.past = 7
        self.k = self.v = np.zeros((rows, hkv, d))
        self.dim = (np.arange(rows)[:, None] * 5 + np.arange(hq)[None, :]) % d
        self.q = np.zeros((rows, hq, d))
        np.put_along_axis(self.q, self.dim[:, :, None], 1.0, axis=2)
        self.S0 = rng.standard_normal((hkv, d, d)).astype(np.float32)

    def out(self, terms=3):
        S = split(self.S0, terms)
        rows, hq, d = self.q.shape
        return np.stack([S[h // (hq // len(S)), self.dim[:, h]] for h in range(hq)], 1)

    def state(self, terms=3):
        return self.S0.astype(np.float64)


class Values:
    """From a zero state; key s is 1 in dim s for the first `live` tokens and 0
    behind them, q is 0: row s of the state after `rows` tokens is
    lam^(rows - 1 - s) v_s.  Decays stay near 1, so lam^n does.

    In one chunk: an exponential, a product, a sum of the tensor cores.  Cut
    into ranges: two exponentials, two products and a sum for the own state of
    the first range; at each further one of `joins` a product with a pair and a
    sum; an exponential and a product in the last chunk."""

    def __init__(self, seed, rows, hq, hkv, d, joins=0):
        rng = np.random.default_rng(seed)
        self.tol = (5 if joins == 0 else 4 + 2 + 2 + 1.1 * joins + 3) * STEP
        self.g = -rng.uniform(1e-4, 4e-4, hkv).astype(np.float32)
        self.scale = 1.0
        self.past = 0
        live = min(rows, 64)
        self.q, self.k = np.zeros((rows, hq, d)), np.zeros((rows, hkv, d))
        self.v = np.zeros((rows, hkv, d))
        self.k[np.arange(live), :, np.arange(live)] = 1
        self.v[:live] = to_bf16(rng.standard_normal((live, hkv, d)))
        self.S0 = np.zeros((hkv, d, d), np.float32)
        self.live = live

    def out(self, terms=3):
        return np.zeros(self.q.shape)

    def state(self, terms=3):
        """The product with the decay is what goes into the tensor cores; in
        64 bits where nothing is left out."""
        rows, hkv, d = self.k.shape
        n = rows - 1 - np.arange(self.live)
        x = np.exp(self.g.astype(np.float64)[:, None] * n)[:, :, None] * self.v[:self.live].transpose(1, 0, 2)
        S = np.zeros((hkv, d, d))
        S[:, :self.live] = x if terms == 3 else split(x, terms)
        return S


def worst(got, want):
    """The largest error of an element, in units of it; exact zeros stay."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    if not np.all(got[want == 0] == 0):
        return np.inf
    at = want != 0
    return float(np.max(np.abs(got[at] - want[at]) / np.abs(want[at]), initial=0.0))
