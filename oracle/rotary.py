"""Rotary-position oracle -- TEST INFRASTRUCTURE ONLY.

Only the tests and ``__graft_entry__.smoke()`` may import this module.  It
shares no code with the CUDA library.

Row element pairs are turned as complex numbers times exp(i angle), in
float64: angle = position of the pair's axis times the pair's frequency.

Parity status: pinned by ``tests/test_oracle_rotary.py`` (closed forms,
lengths, relative positions, the section layouts written out).
"""
from __future__ import annotations

import numpy as np


def axis_of_pairs(sections, interleaved=False):
    """Axis of each pair: sections in order, or dealt in turn to the axes
    that still have pairs to take."""
    left, out, a = list(sections), [], 0
    while sum(left):
        if left[a]:
            left[a] -= 1
            out.append(a)
            if not interleaved and left[a]:
                continue
        a = (a + 1) % len(left)
    return out


def rotate(x, positions, inv_freq, sections=None, interleaved=False, adjacent=False):
    """x float [T][H][d], positions int [axes][T] (or [T]), inv_freq fp32
    [rot/2] -> float64 [T][H][d]."""
    x = np.array(x, dtype=np.float64)
    pos = np.atleast_2d(np.asarray(positions, dtype=np.float64))
    f = np.asarray(inv_freq, dtype=np.float64)
    p = len(f)
    axes = axis_of_pairs(sections if sections is not None else [p], interleaved)
    for i in range(p):
        angle = pos[axes[i]] * f[i]
        e0, e1 = (2 * i, 2 * i + 1) if adjacent else (i, i + p)
        z = (x[:, :, e0] + 1j * x[:, :, e1]) * np.exp(1j * angle)[:, None]
        x[:, :, e0], x[:, :, e1] = z.real, z.imag
    return x
