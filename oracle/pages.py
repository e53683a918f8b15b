"""Plain oracle of the block operators: reserve, fork, free (see include/specverify.h).

Each returns a dict of new arrays and `err`; with err != 0 the arrays are the inputs'.
"""
from __future__ import annotations

import numpy as np

BAD_LENGTH, NO_SPACE, BAD_BLOCK, BAD_SLOT = 8, 16, 32, 128


def _state(**kw):
    return {k: np.array(v) for k, v in kw.items()}


def reserve(block_table, seq_lens, free_stack, free_top, n, *, block_size, num_blocks,
            num_new=None):
    same = _state(block_table=block_table, free_top=free_top)
    s = _state(block_table=block_table, free_top=free_top)
    bt, (B, MB) = s["block_table"], block_table.shape
    err, want = 0, []
    for b in range(B):
        L, m = int(seq_lens[b]), n if num_new is None else int(num_new[b])
        if L < 0 or m < 0 or L + m > MB * block_size:
            err |= BAD_LENGTH
            continue
        for j in range(-(-L // block_size), -(-(L + m) // block_size)):
            if bt[b, j] < -1 or bt[b, j] >= num_blocks:
                err |= BAD_BLOCK
            elif bt[b, j] == -1:
                want.append((b, j))
    top = int(free_top)
    if not err and (top < 0 or top > num_blocks or len(want) > top):
        err = NO_SPACE
    if not err:
        for r, (b, j) in enumerate(want):
            x = int(free_stack[top - 1 - r])
            if x < 0 or x >= num_blocks:
                err = BAD_BLOCK
            bt[b, j] = x
        s["free_top"] = np.array(top - len(want))
    return {**(same if err else s), "err": err}


def fork(block_table, seq_lens, extra_refs, src, dst, free_stack, free_top, *, block_size,
         num_blocks):
    """Also `copies`: (from block, to block, tokens) of every tail block."""
    same = _state(block_table=block_table, seq_lens=seq_lens, extra_refs=extra_refs,
                  free_top=free_top)
    s = {k: v.copy() for k, v in same.items()}
    B, MB = block_table.shape
    bt, sl, refs = s["block_table"], s["seq_lens"], s["extra_refs"]
    top, err, copies = int(free_top), 0, []
    for a, d in zip(src, dst):
        if not (0 <= a < B and 0 <= d < B):
            err |= BAD_SLOT
        elif seq_lens[a] < 0 or seq_lens[a] > MB * block_size or seq_lens[d] != 0:
            err |= BAD_LENGTH
        else:
            for j in range(-(-int(seq_lens[a]) // block_size)):
                x = int(block_table[a, j])
                if x < 0 or x >= num_blocks or block_table[d, j] != -1:
                    err |= BAD_BLOCK
    if not err:
        tails = sum(int(seq_lens[a]) % block_size != 0 for a in src)
        if top < 0 or top > num_blocks or tails > top:
            err = NO_SPACE
    if not err:
        if len(set(map(int, dst))) != len(dst) or set(map(int, dst)) & set(map(int, src)):
            err |= BAD_SLOT
        if any(not 0 <= int(x) < num_blocks for x in free_stack[top - tails:top]):
            err |= BAD_BLOCK
    if not err:
        for a, d in zip(src, dst):
            full, off = divmod(int(seq_lens[a]), block_size)
            for j in range(full):
                bt[d, j] = block_table[a, j]
                refs[block_table[a, j]] += 1
            if off:
                top -= 1
                bt[d, full] = free_stack[top]
                copies.append((int(block_table[a, full]), int(free_stack[top]), off))
            sl[d] = seq_lens[a]
        s["free_top"] = np.array(top)
    return {**(same if err else s), "err": err, "copies": copies}


def free(block_table, seq_lens, extra_refs, rows, free_stack, free_top, *, num_blocks):
    same = _state(block_table=block_table, seq_lens=seq_lens, extra_refs=extra_refs,
                  free_stack=free_stack, free_top=free_top)
    s = {k: v.copy() for k, v in same.items()}
    B = block_table.shape[0]
    top, err = int(free_top), 0
    for r in rows:
        if not 0 <= r < B:
            err |= BAD_SLOT
        elif seq_lens[r] < 0:
            err |= BAD_LENGTH
    if not err:
        if len(set(map(int, rows))) != len(rows):
            err |= BAD_SLOT
        if top < 0 or top > num_blocks:
            err |= BAD_BLOCK
        if any(x < -1 or x >= num_blocks for r in set(map(int, rows)) for x in block_table[r]):
            err |= BAD_BLOCK
    if not err:
        listed = [int(x) for r in rows for x in block_table[r] if x >= 0]
        for x in listed:
            s["extra_refs"][x] -= 1
        if any(s["extra_refs"][x] < -1 for x in listed):
            err = BAD_BLOCK
        order = [x for x in dict.fromkeys(listed) if s["extra_refs"][x] == -1]
        if not err and top + len(order) > num_blocks:
            err = BAD_BLOCK
    if not err:
        for x in order:
            s["free_stack"][top] = x
            s["extra_refs"][x] = 0
            top += 1
        for r in rows:
            s["block_table"][r] = -1
            s["seq_lens"][r] = 0
        s["free_top"] = np.array(top)
    return {**(same if err else s), "err": err}
