"""Attention of rows that share a prefix's blocks against the fp64 oracle, which takes each row by
itself.

Error bound. Cached numbers are exact in the products (e4m3 codes of keys, values widened to bf16,
power-of-two scales), queries down to 2^-9 of their head's largest; smaller ones, fewer than one in
a hundred of these normal numbers, are off by 2^-17 of the largest, so a score by less than 2^-20 of
its sum of magnitudes for them. A score is a sum of 2 D products in fp32; with that it is off by at
most (D + 8) 2^-23 of sum |q_d k_d| * softmax_scale (`reach`; the tensor cores may cut the sum's
terms, hence 2^-23), and a weight by as much of itself; the probability's rounding to bf16 is 2^-8
of each term; exponentials, their argument (2^-24 of an argument that itself is at most twice reach,
in log2 units) and the joins add 2^-19 of the sum of magnitudes (`spread`) at most where reach stays
below 8. Then one rounding to bf16, 2^-8.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from oracle import q8
from tests import q8_helpers as h

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def share(monkeypatch):
    """Most of these cases are too small for sharing to pay: share whatever is common."""
    monkeypatch.setenv("SPECVERIFY_SHARE", "1")


def grouped(rng, groups, own, alone, bs, T, n=None):
    """(L, block_table, starts, members, num_blocks): groups [(prefix, rows)], each row's own
    lengths from own = (lo, hi), `alone` rows in no group, all in a shuffled order."""
    B = sum(r for _, r in groups) + alone
    order = rng.permutation(B)
    L = rng.integers(own[0], own[1] + 1, B)
    shared = np.zeros(B, np.int64)
    members, starts, at = [], [0], 0
    for pre, r in groups:
        rows = order[at:at + r]
        at += r
        L[rows] += pre
        shared[rows] = pre // bs
        members += list(rows)
        starts.append(len(members))
    new = np.full(B, T) if n is None else np.asarray(n)
    held = -(-(L + new) // bs)
    mb = max(1, int(held.max()))
    nb = int((held - shared).clip(0).sum() + sum(p // bs for p, _ in groups)) + 4
    ids = list(rng.permutation(nb))
    bt = np.full((B, mb), -1, np.int64)
    for g, (pre, _) in enumerate(groups):
        blocks = [ids.pop() for _ in range(pre // bs)]
        for r in members[starts[g]:starts[g + 1]]:
            bt[r, :len(blocks)] = blocks
    for b in range(B):
        for j in range(int(shared[b]), int(held[b])):
            bt[b, j] = ids.pop()
    return L, bt, starts, members, nb


def plan_of(bt, L, starts, members, T, Hq, H, bs, nb, n=None, err=None):
    return sv.kv_prefix_plan(h.i32(bt), h.i32(L), h.i32(starts), h.i32(members), tokens=T,
                             q_heads=Hq, kv_heads=H, block_size=bs, num_blocks=nb,
                             num_new=None if n is None else h.i32(n), err_flag=err)


def bound(out, spread, reach, D):
    score = (D + 8) * 2.0 ** -23 * reach
    return ((2.0 ** -8 + 2 * score + 2.0 ** -19 * (1 + reach / 8)) * spread
            + 2.0 ** -8 * np.abs(out) + 1e-30)


def check(got, q, pool, scales, bt, L, n=None, live=None, **kw):
    out, spread, reach = q8.attention(q, pool, scales, bt, L, n, **kw)
    got = got.double().cpu().numpy()
    live = np.ones(len(L), bool) if live is None else live
    off = np.abs(got - out)[live]
    lim = bound(out, spread, reach, q.shape[-1])[live]
    nan = np.isnan(out[live])
    assert (np.isnan(got[live]) == nan).all()
    assert (off <= lim)[~nan].all(), float((off / lim)[~nan].max())


def queries(rng, B, T, Hq, D):
    q = h.bf16_values(rng.normal(size=(B, T, Hq, D)))
    return q, torch.from_numpy(q).bfloat16().cuda()


@pytest.mark.parametrize("groups,own,alone,T,Hq,H,D,bs,more", [
    ([(300, 3)], (1, 40), 0, 5, 8, 2, 128, 16, {}),
    ([(300, 3)], (1, 40), 2, 5, 8, 2, 64, 16, {}),
    ([(127, 2)], (0, 5), 0, 1, 4, 4, 128, 16, {}),           # less than a tile in common
    ([(128, 2)], (0, 0), 0, 1, 4, 4, 128, 16, {}),           # nothing of a row's own but its token
    ([(1000, 7), (200, 2), (513, 4)], (0, 300), 3, 5, 8, 2, 128, 16, {}),
    ([(700, 9)], (1, 200), 1, 7, 28, 4, 128, 32, dict(tree=True)),
    ([(400, 5)], (1, 90), 0, 32, 8, 1, 64, 16, dict(tree=True)),   # 256 queries of a row
    ([(400, 3)], (1, 90), 0, 32, 12, 1, 128, 16, {}),              # 384
    ([(900, 14)], (0, 30), 0, 5, 8, 2, 128, 64, dict(ragged=True)),  # 280: two blocks of queries
    ([(650, 6)], (0, 30), 0, 6, 8, 2, 64, 5, dict(ragged=True)),   # 144: two M tiles; odd blocks
    ([(4000, 2)], (0, 10), 0, 3, 2, 1, 128, 16, {}),         # cut over many CTAs
    ([(5200, 4)], (100, 900), 0, 5, 16, 8, 64, 128, {}),
    ([(2600, 12)], (0, 700), 1, 5, 32, 8, 128, 256, {}),
    ([(40, 1)], (0, 40), 4, 3, 4, 2, 128, 16, {}),           # groups of one
    ([(260, 60)], (0, 20), 4, 2, 2, 2, 64, 16, {}),
])
def test_shared_prefixes(groups, own, alone, T, Hq, H, D, bs, more):
    rng = np.random.default_rng(sum(p * r for p, r in groups) + T)
    B = sum(r for _, r in groups) + alone
    n = rng.integers(0, T + 1, B) if more.get("ragged") else None
    L, bt, starts, members, nb = grouped(rng, groups, own, alone, bs, T, n)
    pool, scales = h.cache(rng, nb, 2, H, bs, D, spread=1)
    pool = h.poison_tails(pool, bt, L + (T if n is None else n), bs)
    q, dq = queries(rng, B, T, Hq, D)
    masks = h.tree_masks(rng, B, T) if more.get("tree") else None
    err = h.i32([0])
    plan = plan_of(bt, L, starts, members, T, Hq, H, bs, nb, n, err)
    out = torch.full_like(dq, 3.0)
    kw = dict(layer=1, num_new=None if n is None else h.i32(n), err_flag=err,
              tree_mask=None if masks is None else h.i32(h.as_int32(masks)))
    args = (dq, h.dev_pool(pool), h.dev_scales(scales), h.i32(bt), h.i32(L), plan)
    sv.kv_q8_prefix_attention(*args, out, **kw)
    assert int(err) == 0
    check(out, q, pool, scales, bt, L, n, layer=1, tree_mask=masks)
    again = torch.full_like(dq, 5.0)
    sv.kv_q8_prefix_attention(*args, again, **kw)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def _small(seed=0, T=4, Hq=8, H=2, D=128, bs=16, groups=((500, 3), (300, 2)), own=(1, 60), alone=1):
    rng = np.random.default_rng(seed)
    L, bt, starts, members, nb = grouped(rng, list(groups), own, alone, bs, T)
    pool, scales = h.cache(rng, nb, 1, H, bs, D, spread=1)
    q, dq = queries(rng, len(L), T, Hq, D)
    return rng, L, bt, starts, members, nb, pool, scales, q, dq


def _run(dq, pool, scales, bt, L, plan, **kw):
    out = torch.full_like(dq, 3.0)
    sv.kv_q8_prefix_attention(dq, h.dev_pool(pool), h.dev_scales(scales), h.i32(bt), h.i32(L),
                              plan, out, **kw)
    return out


def test_groups_are_a_guess():
    """Rows that share nothing, rows that share less than their group, one listed twice, rows out
    of range: the time changes, the result does not."""
    rng, L, bt, starts, members, nb, pool, scales, q, dq = _small()
    B = len(L)
    for st, mem, bits in (([0, B], rng.permutation(B), 0), ([0, 2, 2, B], np.arange(B), 0),
                          (starts, members[:1] + members[:4], sv.SPEC_DERR_BAD_SLOT),
                          ([1, 5], [99, *members[:3], -1], sv.SPEC_DERR_BAD_SLOT),
                          ([0, 4, 2], members[:5], sv.SPEC_DERR_BAD_SLOT),
                          ([-1, 3], members[:5], sv.SPEC_DERR_BAD_SLOT),
                          ([0, 6], members[:5], sv.SPEC_DERR_BAD_SLOT)):
        err = h.i32([0])
        plan = plan_of(bt, L, st, mem, 4, 8, 2, 16, nb, err=err)
        out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == bits
        check(out, q, pool, scales, bt, L)


def test_plan_of_other_lengths_or_sizes():
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(1)
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb)
    moved = L.copy()
    moved[2] += 1
    bt2 = np.concatenate([bt, np.full((len(L), 1), -1)], 1)
    err = h.i32([0])
    out = _run(dq, pool, scales, bt, moved, plan, err_flag=err)
    assert int(err) == sv.SPEC_DERR_BAD_LENGTH and torch.isnan(out[2]).all()
    live = np.arange(len(L)) != 2
    check(out, q, pool, scales, bt, L, live=live)
    for other, kw in ((plan_of(bt, L, starts, members, 3, 8, 2, 16, nb), {}),
                      (plan_of(bt2, L, starts, members, 4, 8, 2, 16, nb), {}),
                      (torch.zeros(4096, dtype=torch.uint8, device="cuda"), {}),
                      (plan[:plan.numel() - 512], {})):
        err = h.i32([0])
        out = _run(dq, pool, scales, bt, L, other, err_flag=err)
        assert int(err) == sv.SPEC_DERR_BAD_SLOT and torch.isnan(out).all()


def test_bad_lengths_and_blocks():
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(2)
    n = np.full(len(L), 4)
    a, b = members[0], members[3]         # of the two groups
    L[a], n[b] = -1, 5                    # both invalid; their groups go on without them
    c = members[1]
    bt[c, int(L[c]) // 16] = nb + 7       # the block of its new tokens
    err = h.i32([0])
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb, n, err)
    assert int(err) == 0
    out = _run(dq, pool, scales, bt, L, plan, num_new=h.i32(n), err_flag=err)
    assert int(err) == sv.SPEC_DERR_BAD_LENGTH | sv.SPEC_DERR_BAD_BLOCK
    assert torch.isnan(out[a]).all() and torch.isnan(out[b]).all()
    check(out, q, pool, scales, bt, L, n)
    # the whole group's prefix has a bad block: what sees it is NaN, whoever reads it
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(2)
    bt[members[:3], 10] = -1
    err = h.i32([0])
    out = _run(dq, pool, scales, bt, L, plan_of(bt, L, starts, members, 4, 8, 2, 16, nb),
               err_flag=err)
    assert int(err) == sv.SPEC_DERR_BAD_BLOCK and torch.isnan(out[members[:3]]).all()
    check(out, q, pool, scales, bt, L)


def test_scales_that_are_not_plain():
    """Scales past 2^7, below 2^-100, zero and between powers of two; a NaN scale is a NaN key."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(3)
    rng = np.random.default_rng(3)
    kinds = rng.integers(0, 5, scales.shape)
    scales[:, :, 1] = np.select([kinds == 0, kinds == 1, kinds == 2, kinds == 3],
                                [2.0 ** 9, 0.0, 2.0 ** -103, 1.5 * 2.0 ** -4], 0.25)[:, :, 1]
    scales = scales.astype(np.float32).astype(np.float64)
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb)
    out = _run(dq, pool, scales, bt, L, plan)
    want, spread, reach = q8.attention(q, pool, scales, bt, L)
    # code * scale is rounded to bf16 where the scale is no power of two: once more 2^-8
    lim = bound(want, spread, reach, 128) + 2.0 ** -8 * spread
    assert (np.abs(out.double().cpu().numpy() - want) <= lim).all()
    x = int(bt[members[0], 3])
    scales[x, 0, 0, 1] = np.nan
    out = _run(dq, pool, scales, bt, L, plan)
    hit = [r for r in range(len(L)) if bt[r, 3] == x]
    assert torch.isnan(out[hit][:, :, 4:]).all() and not torch.isnan(out[hit][:, :, :4]).any()
    rest = [r for r in range(len(L)) if r not in hit]
    assert not torch.isnan(out[rest]).any()


def test_rising_and_large_scores():
    """Keys that grow along the sequence move the references again and again; scores of a few
    hundred leave one key with all the weight."""
    rng, L, bt, starts, members, nb, pool, scales, q, dq = _small(4, groups=((1500, 4), (700, 3)))
    order = np.zeros(nb)
    for g in range(2):
        for r in members[starts[g]:starts[g + 1]]:
            for j, x in enumerate(bt[r]):
                if x >= 0:
                    order[x] = j
    scales[:, :, 0] = 2.0 ** (-8 + np.clip(order, 0, 100) // 12)[:, None, None]
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb)
    out = _run(dq, pool, scales, bt, L, plan)
    check(out, q, pool, scales, bt, L)
    q[1, 2, 3] = np.nan
    out = _run(torch.from_numpy(q).bfloat16().cuda(), pool, scales, bt, L, plan)
    assert torch.isnan(out[1, 2, 3]).all() and int(torch.isnan(out).sum()) == 128


@pytest.mark.parametrize("dtype,D", [(torch.float32, 128), (torch.bfloat16, 96)])
def test_other_types_and_heads(dtype, D):
    """What the shared form does not take: each row by itself, the same result."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(5, D=D)
    dq = dq.to(dtype)
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb)
    out = _run(dq, pool, scales, bt, L, plan)
    want = torch.empty_like(dq)
    sv.kv_q8_attention(dq, h.dev_pool(pool), h.dev_scales(scales), h.i32(bt), h.i32(L), want)
    assert torch.equal(out, want)


def test_after_fork_and_on_streams_and_captured():
    """Tables as kv_fork leaves them; the calls on another stream, captured, and replayed with
    lengths that have moved on, next to eager calls."""
    rng = np.random.default_rng(6)
    bs, T, Hq, H, D, F = 16, 3, 8, 2, 64, 5
    L0 = 333
    bt, left, nb = h.table(rng, [L0 + T], bs, max_blocks=40, spare=80)
    pool, scales = h.cache(rng, nb, 1, H, bs, D, spread=1)
    table = h.i32(np.concatenate([bt, np.full((F, 40), -1)]))
    table[0, -(-L0 // bs):] = -1
    lens = h.i32([L0] + [0] * F)
    dp, ds = h.dev_pool(pool), h.dev_scales(scales)
    free, top, status = h.i32(np.pad(left, (0, nb - len(left)))), h.i32([len(left)]), h.i32([0])
    refs = h.i32(np.zeros(nb))
    sv.kv_fork(table, lens, refs, h.i32([0] * F), h.i32(range(1, F + 1)), dp, free, top, status,
               block_size=bs, kv_scales=ds)
    sv.kv_reserve(table, lens, free, top, status, n=T + 20, block_size=bs, num_blocks=nb)
    assert int(status) == 0
    B = F + 1
    q, dq = queries(rng, B, T, Hq, D)
    k = torch.from_numpy(rng.normal(size=(B, T, H, D))).bfloat16().cuda()
    starts, members = h.i32([0, B]), h.i32(range(B))
    err = h.i32([0])

    def step(out, stream=None):
        sv.kv_q8_append(k, k, dp, ds, table, lens, stream=stream, err_flag=err)
        plan = sv.kv_prefix_plan(table, lens, starts, members, tokens=T, q_heads=Hq, kv_heads=H,
                                 block_size=bs, num_blocks=nb, stream=stream, err_flag=err)
        sv.kv_q8_prefix_attention(dq, dp, ds, table, lens, plan, out, stream=stream, err_flag=err)

    def expect(out):
        torch.cuda.synchronize()
        assert int(err) == 0
        check(out, q, dp.view(torch.uint8).cpu().numpy(), ds.double().cpu().numpy(),
              table.cpu().numpy(), lens.cpu().numpy())

    out = torch.empty_like(dq)
    step(out)
    expect(out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = torch.empty_like(dq)
    step(other, side)
    side.synchronize()
    assert torch.equal(other, out)
    graph, captured = torch.cuda.CUDAGraph(), torch.empty_like(dq)
    with torch.cuda.graph(graph):
        step(captured)
    for _ in range(3):
        lens += T
        graph.replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
        expect(captured)
        step(out)
        expect(out)
        assert torch.equal(out, captured)


def test_a_wait_runs_out(monkeypatch):
    """One row's values withheld: the call reports it and returns, the next call is as ever."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(7, groups=((900, 12), (300, 2)))
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb)
    err = h.i32([0])
    monkeypatch.setenv("SPECVERIFY_STALL_ROW", "3")
    monkeypatch.setenv("SPECVERIFY_IDLE_NS", "5000000")
    _run(dq, pool, scales, bt, L, plan, err_flag=err)
    assert int(err) == sv.SPEC_DERR_TIMEOUT
    # the row with which a group begins: its shared keys as well
    err = h.i32([0])
    monkeypatch.setenv("SPECVERIFY_STALL_ROW", str(int(members[0])))
    _run(dq, pool, scales, bt, L, plan, err_flag=err)
    assert int(err) == sv.SPEC_DERR_TIMEOUT
    monkeypatch.delenv("SPECVERIFY_STALL_ROW")
    monkeypatch.delenv("SPECVERIFY_IDLE_NS")
    err = h.i32([0])
    out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
    assert int(err) == 0
    check(out, q, pool, scales, bt, L)
