"""fp64 NumPy oracle of the norms and rotary positions of queries and keys, and of the same with
keys and values appended to the 8-bit paged cache. Written from the definitions in
include/specverify.h, head by head.
"""
from __future__ import annotations

import numpy as np

from oracle import q8


def heads(x, weight, positions, inv_freq, *, interleaved=False, factor=1.0, eps=1e-6):
    """(y, reach) of x [B, T, H, D]: y the normed and turned heads in fp64; reach the sum of the
    magnitudes that each number was made from, for error bounds. inv_freq as fp32 holds it."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    reach = np.abs(y)
    P = 0 if inv_freq is None else len(inv_freq)
    for i in range(P):
        ang = np.asarray(positions, np.float64)[..., None] * np.float64(inv_freq[i])
        c, s = factor * np.cos(ang), factor * np.sin(ang)
        at, to = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
        a, b = y[..., at].copy(), y[..., to].copy()
        y[..., at], y[..., to] = a * c - b * s, b * c + a * s
        reach[..., at] = reach[..., to] = (np.abs(a) + np.abs(b)) * abs(factor)
    return y, reach


def append(k, v, pool, scales, block_table, seq_lens, num_new=None, *, layer=0, **turn):
    """kv_q8_norm_rope_append's cache: q8.append of the normed and turned keys, and their reach."""
    y, reach = heads(k, turn.pop("weight"), turn.pop("positions"), turn.pop("inv_freq"), **turn)
    return (*q8.append(y, v, pool, scales, block_table, seq_lens, num_new, layer=layer), y, reach)
