"""fp64 restatement of ragged attention over a paged cache: causal (a
sequence's newest tokens over its cache) and cross (a decoder's tokens over
an encoder's states).

Token i of sequence b's nq query tokens (rows q_start[b] .. q_start[b + 1])
sees the first n - nq + i + 1 cached tokens (causal) or all n (cross):
softmax(scale q.K) V over those, zeros when there are none.
"""
from __future__ import annotations

import numpy as np

from . import paged_attention as PA


def _rows(cache, scale, table, n, g):
    bs = cache.shape[2]
    x = PA.gather_sequence(cache[:, g:g + 1], table, n, bs)[:, 0]
    if scale is not None:
        x = PA.dequant_rows(x, scale[np.asarray(table)[np.arange(n) // bs], g])
    return x.astype(np.float64)


def attend_rows(q, k_cache, v_cache, tables, q_start, lens, scale, causal, k_scale=None,
                v_scale=None):
    """(out, spread): out [T, Hq, d] in fp64, NaN at rows of no sequence;
    spread [T, Hq, d] = sum_t softmax_t |V_t|, what an error of the weights
    is measured by."""
    T, hq, d = q.shape
    hkv = k_cache.shape[1]
    group = hq // hkv
    out = np.full((T, hq, d), np.nan)
    spread = np.full((T, hq, d), np.nan)
    for b, n in enumerate(lens):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        if hi == lo:
            continue
        out[lo:hi] = 0.0
        spread[lo:hi] = 0.0
        if n == 0:
            continue
        for g in range(hkv):
            k = _rows(k_cache, k_scale, tables[b], n, g)
            v = _rows(v_cache, v_scale, tables[b], n, g)
            for h in range(g * group, (g + 1) * group):
                s = scale * (q[lo:hi, h].astype(np.float64) @ k.T)
                if causal:
                    place = n - (hi - lo) + np.arange(hi - lo)
                    s[np.arange(n)[None, :] > place[:, None]] = -np.inf
                w = np.exp(s - s.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[lo:hi, h] = w @ v
                spread[lo:hi, h] = w @ np.abs(v)
    return out, spread
