"""The way of a step's queries, keys and values through the operators, as they are used together
(reserve, norms and positions into the cache, plan, attention of shared prefixes, verification,
commit, release), and what the shared form's other tests do not reach. Each against the fp64
oracles; the bounds are those of test_gpu_norm_rope.py and test_gpu_prefix.py."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from oracle import rope
from tests import q8_helpers as h
from tests.test_gpu_norm_rope import _bound
from tests.test_gpu_prefix import _run, _small, check, grouped, plan_of, queries, share  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,H,D,tree,L0", [(5, 8, 2, 128, False, (700, 90)),
                                              (7, 8, 1, 64, True, (260, 1000)),
                                              (1, 4, 4, 128, False, (128, 3))])
def test_steps_of_forked_rows(T, Hq, H, D, tree, L0):
    rng = np.random.default_rng(T)
    bs, F, V, B = 16, 4, 512, 2 + 2 * 4
    mb = max(L0) // bs + 8
    nb = sum(-(-x // bs) for x in L0) + 100
    bt, left, _ = h.table(rng, L0, bs, max_blocks=mb, spare=100)
    pool, scales = h.cache(rng, nb, 1, H, bs, D, spread=1)
    table = h.i32(np.concatenate([bt, np.full((2 * F, mb), -1)]))
    lens, refs = h.i32([*L0] + [0] * 2 * F), h.i32(np.zeros(nb))
    dp, ds = h.dev_pool(pool), h.dev_scales(scales)
    free, top, status = h.i32(np.pad(left, (0, nb - len(left)))), h.i32([len(left)]), h.i32([0])
    err = h.i32([0])
    dst = np.arange(2, B)
    sv.kv_fork(table, lens, refs, h.i32(dst % 2), h.i32(dst), dp, free, top, status,
               block_size=bs, kv_scales=ds)
    starts, members = h.i32([0, F + 1, B]), h.i32([*range(0, B, 2), *range(1, B, 2)])
    f = sv.rope_frequencies(D // 2, 10000.0)[0]
    w = torch.from_numpy(1 + 0.3 * rng.normal(size=(2, D))).bfloat16().cuda()
    wn = w.double().cpu().numpy()
    masks = h.tree_masks(rng, B, T) if tree else None
    tm = None if masks is None else h.i32(h.as_int32(masks))
    for _ in range(3):
        L = lens.cpu().numpy()
        depth = np.zeros((B, T), np.int64)
        if tree:
            depth = np.array([[bin(int(m)).count("1") - 1 for m in row] for row in masks])
        pos = L[:, None] + (depth if tree else np.arange(T))
        x = torch.from_numpy(rng.normal(size=(B, T, Hq + 2 * H, D))).bfloat16().cuda()
        q, k, v = x.split([Hq, H, H], 2)
        qo, out = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
        sv.kv_reserve(table, lens, free, top, status, n=T, block_size=bs, num_blocks=nb)
        before = dp.view(torch.uint8).cpu().numpy(), ds.double().cpu().numpy()
        sv.kv_q8_norm_rope_append(q, k, v, qo, dp, ds, table, lens, inv_freq=f, q_weight=w[0],
                                  k_weight=w[1], positions=h.i32(pos) if tree else None,
                                  err_flag=err)
        plan = sv.kv_prefix_plan(table, lens, starts, members, tokens=T, q_heads=Hq, kv_heads=H,
                                 block_size=bs, num_blocks=nb, err_flag=err)
        sv.kv_q8_prefix_attention(qo, dp, ds, table, lens, plan, out, tree_mask=tm, err_flag=err)
        assert int(err) == 0 and int(status) == 0
        y, reach = rope.heads(q.double().cpu().numpy(), wn[0], pos, f.cpu().numpy())
        qn = qo.double().cpu().numpy()
        assert (np.abs(qn - y) <= _bound(y, reach, pos, "bf16")).all()
        codes, sc = dp.view(torch.uint8).cpu().numpy(), ds.double().cpu().numpy()
        t = table.cpu().numpy()
        want, wsc, *_ = rope.append(k.double().cpu().numpy(), v.double().cpu().numpy(), *before, t,
                                    L, weight=wn[1], positions=pos, inv_freq=f.cpu().numpy())
        assert np.array_equal(codes[:, :, 1], want[:, :, 1])
        assert np.array_equal(sc[:, :, 1], wsc[:, :, 1])
        check(out, qn, codes, sc, t, L, tree_mask=masks)
        if tree or T == 1:  # one token is kept: no drafts, or none accepted
            acc, K = torch.zeros(B, dtype=torch.int32, device="cuda"), 0
        else:
            K = T - 1
            logits = torch.from_numpy(rng.normal(size=(B, T, V))).float().cuda()
            drafts = logits[:, :K].argmax(-1).int()
            drafts[::3, 1] = (drafts[::3, 1] + 1) % V
            acc = torch.empty(B, dtype=torch.int32, device="cuda")
            sv.spec_verify_greedy(logits, drafts, torch.empty((B, T), dtype=torch.int32,
                                                              device="cuda"), acc)
            assert acc.tolist() == [1 if b % 3 == 0 else K for b in range(B)]
        sv.kv_commit_inplace(table, lens, acc, free, top, status, K=K, block_size=bs,
                             num_blocks=nb)
        assert np.array_equal(lens.cpu().numpy(), L + acc.cpu().numpy() + 1)
    sv.kv_free(table, lens, refs, h.i32(rng.permutation(B)), free, top, status, num_blocks=nb)
    assert int(status) == 0 and not refs.any()


@pytest.mark.parametrize("T,Hq,H,D,bs", [
    (10, 16, 2, 128, 16),   # 80 queries of a row and head: an M tile each, 400 of the group
    (17, 8, 2, 64, 32),     # 68
    (32, 16, 1, 128, 16),   # 512 of a row: two blocks of 256
    (9, 56, 2, 128, 48),    # 252, groups of 28 heads
])
def test_many_queries_of_a_row(T, Hq, H, D, bs):
    rng = np.random.default_rng(Hq)
    groups, alone = [(300, 5), (140, 2)], 1
    n = rng.integers(0, T + 1, 8)
    L, bt, starts, members, nb = grouped(rng, groups, (0, 170), alone, bs, T, n)
    pool, scales = h.cache(rng, nb, 1, H, bs, D, spread=1)
    q, dq = queries(rng, 8, T, Hq, D)
    plan = plan_of(bt, L, starts, members, T, Hq, H, bs, nb, n)
    err = h.i32([0])
    out = _run(dq, pool, scales, bt, L, plan, num_new=h.i32(n), err_flag=err)
    assert int(err) == 0
    check(out, q, pool, scales, bt, L, n)


def test_signs_of_scales():
    """K scales below zero, V scales below zero."""
    rng, L, bt, starts, members, nb, pool, scales, q, dq = _small(11)
    scales = scales * rng.choice([-1.0, 1.0], scales.shape)
    out = _run(dq, pool, scales, bt, L, plan_of(bt, L, starts, members, 4, 8, 2, 16, nb))
    check(out, q, pool, scales, bt, L)


@pytest.mark.parametrize("n", [[0] * 6, [0, 0, 0, 0, 4, 0], [0, 3, 0, 0, 0, 0]])
def test_rows_without_new_tokens(n):
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(12)
    n = np.array(n)
    err = h.i32([0])
    plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb, n, err)
    out = _run(dq, pool, scales, bt, L, plan, num_new=h.i32(n), err_flag=err)
    assert int(err) == 0 and not out[n == 0].any()
    check(out, q, pool, scales, bt, L, n)


def test_no_groups():
    _, L, bt, _, _, nb, pool, scales, q, dq = _small(13)
    err = h.i32([0])
    for starts, members in (([0], []), ([0, 0], []), ([0], [2, 3])):
        plan = plan_of(bt, L, starts, members, 4, 8, 2, 16, nb, err=err)
        out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == 0
        check(out, q, pool, scales, bt, L)


def test_what_is_shared(monkeypatch):
    """By itself a plan shares where that saves time: rows that it leaves alone have the bytes that
    kv_q8_attention gives them, and a plan that shares nothing all of them."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(16, groups=((500, 3), (300, 2)))
    want = torch.empty_like(dq)
    sv.kv_q8_attention(dq, h.dev_pool(pool), h.dev_scales(scales), h.i32(bt), h.i32(L), want)
    out = _run(dq, pool, scales, bt, L, plan_of(bt, L, starts, members, 4, 8, 2, 16, nb))
    alone = [r for r in range(len(L)) if r not in members]
    assert torch.equal(out[alone], want[alone]) and not torch.equal(out, want)
    monkeypatch.delenv("SPECVERIFY_SHARE")
    out = _run(dq, pool, scales, bt, L, plan_of(bt, L, starts, members, 4, 8, 2, 16, nb))
    assert torch.equal(out, want)
    # its lists are looked at all the same
    for st, mem in (([0, 4, 2], members), (starts, [99, *members[1:]]), ([0, 5], [members[0]] * 5)):
        err = h.i32([0])
        plan = plan_of(bt, L, st, mem, 4, 8, 2, 16, nb, err=err)
        assert int(err) == sv.SPEC_DERR_BAD_SLOT
        assert torch.equal(_run(dq, pool, scales, bt, L, plan), want)
    # tables long enough to share much, rows that do not
    wide = np.concatenate([bt, np.full((len(L), 20000), -1)], 1)
    out = _run(dq, pool, scales, wide, L, plan_of(wide, L, starts, members, 4, 8, 2, 16, nb))
    assert torch.equal(out, want)
    # 64 rows behind 12000 common tokens
    rng = np.random.default_rng(16)
    L, bt, starts, members, nb = grouped(rng, [(12000, 64)], (0, 100), 2, 16, 2)
    pool, scales = h.cache(rng, nb, 1, 2, 16, 64, spread=1)
    q, dq = queries(rng, 66, 2, 32, 64)
    args = bt, L, starts, members, 2, 32, 2, 16, nb
    out = _run(dq, pool, scales, bt, L, plan_of(*args))
    check(out, q, pool, scales, bt, L)
    monkeypatch.setenv("SPECVERIFY_SHARE", "1")
    assert torch.equal(out, _run(dq, pool, scales, bt, L, plan_of(*args)))


def test_first_tokens():
    """Rows of length zero, by themselves and in a group; one token of one row."""
    rng = np.random.default_rng(14)
    for T, lens in ((1, [0]), (3, [0, 0, 5, 0, 130])):
        L = np.array(lens)
        bt, _, nb = h.table(rng, L + T, 16)
        pool, scales = h.cache(rng, nb, 1, 2, 16, 128, spread=1)
        q, dq = queries(rng, len(L), T, 8, 128)
        err = h.i32([0])
        plan = plan_of(bt, L, [0, len(L)], range(len(L)), T, 8, 2, 16, nb, err=err)
        out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == 0
        check(out, q, pool, scales, bt, L)


def test_a_pool_past_32_bits():
    """Blocks whose bytes lie beyond 4 GiB: the append's and the attention's offsets."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(15)
    big = (9 << 29) // pool[0].size + nb            # blocks of 4.5 GiB, and these
    up = big - nb
    dp = torch.zeros((big, *pool.shape[1:]), dtype=torch.uint8, device="cuda")
    ds = torch.zeros((big, *scales.shape[1:]), device="cuda")
    dp[up:], ds[up:] = torch.from_numpy(pool).cuda(), h.dev_scales(scales)
    high = np.where(bt >= 0, bt + up, bt)
    B, err = len(L), h.i32([0])
    rng = np.random.default_rng(15)
    k = torch.from_numpy(rng.normal(size=(B, 4, 2, 128))).bfloat16().cuda()
    q0 = torch.empty_like(dq)
    f = sv.rope_frequencies(64, 10000.0)[0]
    dp = dp.view(torch.float8_e4m3fn)
    sv.kv_q8_norm_rope_append(dq, k, k, q0, dp, ds, h.i32(high), h.i32(L), inv_freq=f, err_flag=err)
    plan = plan_of(high, L, starts, members, 4, 8, 2, 16, big, err=err)
    out = torch.empty_like(dq)
    sv.kv_q8_prefix_attention(q0, dp, ds, h.i32(high), h.i32(L), plan, out, err_flag=err)
    assert int(err) == 0
    codes = dp.view(torch.uint8)
    assert not codes[:up].any()
    check(out, q0.double().cpu().numpy(), codes[up:].cpu().numpy(), ds[up:].double().cpu().numpy(),
          bt, L)
