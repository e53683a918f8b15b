"""fp64 NumPy oracle of the 8-bit paged cache: format, appending, attention.

A block of tokens and head holds e4m3 codes and one power-of-two scale; a number is
code * scale. Written from the definitions in include/specverify.h, row by row.
"""
from __future__ import annotations

import numpy as np

MAX = 448.0
MIN_EXP = -100


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: 1 sign bit, 4 exponent bits (bias 7), 3 bits of
    fraction; exponent 0 is subnormal, the codes 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


VALUES = e4m3_values()


def encode(x: np.ndarray) -> np.ndarray:
    """Codes of x: nearest, ties to the even code, magnitudes over 448 become 448."""
    x = np.asarray(x, np.float64)
    grid = VALUES[:127]
    a = np.minimum(np.abs(x), MAX)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(amax: float) -> float:
    """The smallest 2^e, e >= -100, with amax <= 448 * 2^e."""
    e = MIN_EXP
    while amax > MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(k, v, pool, scales, block_table, seq_lens, num_new=None, *, layer=0):
    """pool uint8 [NB, NL, 2, H, bs, D], scales fp64 [NB, NL, 2, H]: new copies after
    appending, and the error bits. k, v [B, T, H, D]; inf and NaN as the header says."""
    pool, scales = pool.copy(), scales.copy()
    NB, _, _, H, bs, _ = pool.shape
    B, T = k.shape[:2]
    big = float(np.finfo(np.float32).max)
    err = 0
    for b in range(B):
        L, n = int(seq_lens[b]), T if num_new is None else int(num_new[b])
        if L < 0 or n < 0 or n > T or L + n > block_table.shape[1] * bs:
            err |= 8
            continue
        at = L
        while at < L + n:
            o = at % bs
            m = min(bs - o, L + n - at)
            x = int(block_table[b, at // bs])
            if x < 0 or x >= NB:
                err |= 32
            else:
                for plane, src in enumerate((k, v)):
                    for h in range(H):
                        new = src[b, at - L:at - L + m, h].astype(np.float64)
                        if not np.isfinite(new).all():
                            err |= 256
                        new = np.clip(np.where(np.isnan(new), 0.0, new), -big, big)
                        s = block_scale(float(np.abs(new).max()))
                        if o:
                            was = scales[x, layer, plane, h]
                            s = max(s, was)
                            if s != was:
                                old = VALUES[pool[x, layer, plane, h, :o]]
                                pool[x, layer, plane, h, :o] = encode(old * (was / s))
                        pool[x, layer, plane, h, o:o + m] = encode(new / s)
                        scales[x, layer, plane, h] = s
            at += m
    return pool, scales, err


def visible(L, n, T, *, window=0, sinks=0, tree_mask=None):
    """[T, L + n] truth values: which keys each query sees. tree_mask: [T] integers."""
    see = np.zeros((T, L + n), bool)
    for t in range(n):
        for j in range(L + n):
            if tree_mask is not None:
                see[t, j] = j < L or (int(tree_mask[t]) >> (j - L)) & 1
            else:
                see[t, j] = j <= L + t and (window == 0 or j > L + t - window or j < sinks)
    return see


def attention(q, pool, scales, block_table, seq_lens, num_new=None, *, layer=0,
              softmax_scale=None, window=0, sinks=0, tree_mask=None):
    """(out [B, T, Hq, D], spread): out the attention in fp64, spread = sum_j w_j |v_j| and
    reach = the largest sum_d |q_d k_d| * softmax_scale of the query, for error bounds."""
    B, T, Hq, D = q.shape
    NB, _, _, H, bs, _ = pool.shape
    G = Hq // H
    sc = D ** -0.5 if softmax_scale is None else softmax_scale
    out = np.zeros(q.shape)
    spread = np.zeros(q.shape)
    reach = np.zeros((B, T, Hq, 1))
    for b in range(B):
        L, n = int(seq_lens[b]), T if num_new is None else int(num_new[b])
        if L < 0 or n < 0 or n > T or L + n > block_table.shape[1] * bs:
            out[b] = np.nan
            continue
        if n == 0:
            continue
        pages = block_table[b, :-(-(L + n) // bs)].astype(int)
        good = (pages >= 0) & (pages < NB)
        pg = np.where(good, pages, 0)
        kv = VALUES[pool[pg, layer]] * scales[pg, layer][..., None, None]  # [P, 2, H, bs, D]
        kv = np.where(good[:, None, None, None, None], kv, np.nan)
        kv = kv.transpose(1, 2, 0, 3, 4).reshape(2, H, -1, D)[:, :, :L + n]
        see = visible(L, n, T, window=window, sinks=sinks,
                      tree_mask=None if tree_mask is None else tree_mask[b])
        for t in range(n):
            js = np.nonzero(see[t])[0]
            if len(js) == 0:
                continue
            for hq in range(Hq):
                k, v = kv[0, hq // G, js], kv[1, hq // G, js]
                x = q[b, t, hq].astype(np.float64)
                z = (k @ x) * sc
                w = np.exp(z - np.max(z))
                w /= w.sum()
                out[b, t, hq] = w @ v
                spread[b, t, hq] = w @ np.abs(v)
                reach[b, t, hq] = np.max(np.abs(k) @ np.abs(x)) * sc
    return out, spread, reach
