"""Linear-attention oracle -- TEST INFRASTRUCTURE ONLY.

Only the tests and ``__graft_entry__.smoke()`` may import this module.  It
shares no code with the CUDA library.

The recurrence as it is defined, token by token, in float64:
    S <- exp(log_decay) S + k v^T,   out = scale * q^T S
with one state per (sequence, kv head) and q head h reading kv head
h // (Hq / Hkv).

Parity status: pinned by ``tests/test_oracle_linear.py`` (the closed double
sum, closed forms, chunk splits, linearity in v).
"""
from __future__ import annotations

import numpy as np


def attend(states, log_decay, q, k, v, query_start_loc, state_slots, context_lens, scale, new_slots=None):
    """states float [slots][Hkv][d][d] (k index, v index); returns (out
    float64 [T][Hq][d], states after the call as float64).  Sequences that
    the library skips give zero rows; rows behind the last are NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    before = np.array(states, dtype=np.float64)
    after = before.copy()
    new_slots = state_slots if new_slots is None else new_slots
    T, hq, d = q.shape
    hkv = k.shape[1]
    lam = np.exp(np.asarray(log_decay, dtype=np.float64))
    out = np.full((T, hq, d), np.nan)
    for s in range(len(context_lens)):
        r0, r1 = int(query_start_loc[s]), int(query_start_loc[s + 1])
        n, rows = int(context_lens[s]), r1 - r0
        if rows == 0:
            continue
        load, store = int(state_slots[s]), int(new_slots[s])
        goes_on = n > rows
        if n < rows or store >= len(before) or (goes_on and not 0 <= load < len(before)):
            out[r0:r1] = 0.0
            continue
        S = before[load].copy() if goes_on else np.zeros((hkv, d, d))
        for t in range(r0, r1):
            for g in range(hkv):
                S[g] = lam[g] * S[g] + np.outer(k[t, g], v[t, g])
            for h in range(hq):
                out[t, h] = scale * (q[t, h] @ S[h // (hq // hkv)])
        if store >= 0:
            after[store] = S
    return out, after
