"""Seeded inputs of the 8-bit cache tests, and device copies of them."""
import numpy as np


def i32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def table(rng, lengths, bs, max_blocks=None, spare=5):
    """(block_table [B, MB], ids left over, num_blocks): shuffled blocks for `lengths` tokens."""
    held = [-(-int(n) // bs) for n in lengths]
    mb = max(1, max(held)) if max_blocks is None else max_blocks
    nb = sum(held) + spare
    ids = rng.permutation(nb)
    bt = np.full((len(held), mb), -1, np.int64)
    at = 0
    for b, h in enumerate(held):
        bt[b, :h] = ids[at:at + h]
        at += h
    return bt, ids[at:], nb


def cache(rng, nb, layers, heads, bs, dim, spread=3):
    """Codes of normal numbers and power-of-two scales over 2 * spread + 1 binades; the codes
    after a row's end are NaN in half of the blocks, as memory that nobody wrote may be."""
    import oracle.q8 as q8
    pool = q8.encode(rng.normal(0, 60, (nb, layers, 2, heads, bs, dim)))
    scales = 2.0 ** rng.integers(-6 - spread, -6 + spread + 1, (nb, layers, 2, heads))
    return pool, scales


def poison_tails(pool, bt, ends, bs):
    """NaN codes in every slot past the rows' ends, and in blocks that no row holds."""
    pool = pool.copy()
    held = set()
    for b, n in enumerate(ends):
        for j in range(-(-int(n) // bs)):
            x = int(bt[b, j])
            if 0 <= x < len(pool):
                held.add(x)
                if (j + 1) * bs > n:
                    pool[x, :, :, :, int(n) - j * bs:] = 0x7f
    for x in set(range(len(pool))) - held:
        pool[x] = 0xff
    return pool


def dev_pool(pool):
    import torch
    return torch.from_numpy(pool.copy()).cuda().view(torch.float8_e4m3fn)


def dev_scales(scales):
    import torch
    return torch.from_numpy(scales.astype(np.float32)).cuda()


def bf16_values(x):
    """x rounded to bf16, as fp64."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def tree_masks(rng, B, T):
    m = np.zeros((B, T), np.int64)
    m[:, 0] = 1
    for t in range(1, T):
        p = rng.integers(0, t, size=B)
        m[:, t] = m[np.arange(B), p] | (1 << t)
    return m


def as_int32(m):
    return np.where(m >= 1 << 31, m - (1 << 32), m)
