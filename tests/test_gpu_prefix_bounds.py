"""Attention of shared prefixes at the ends of its domain: waits that run out while products are in
flight, numbers near the ends of fp32, codes that are no numbers, the largest lists. The bounds are
those of test_gpu_prefix.py."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from oracle import q8
from tests import q8_helpers as h
from tests.test_gpu_prefix import (_run, _small, bound, check, grouped, plan_of, queries,
                                   share)  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T,groups", [(128, 4, ((5000, 40), (2000, 24))),   # two M tiles
                                        (64, 4, ((5000, 40), (2000, 24))),
                                        (128, 1, ((5000, 9), (2000, 5)))])    # one, in turns
def test_waits_run_out_with_products_in_flight(monkeypatch, D, T, groups):
    """The second group's keys are withheld where CTAs have the first group's products in flight:
    what is issued ends before the CTA does, and the next call is as ever."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(21, T=T, D=D, groups=groups)
    plan = plan_of(bt, L, starts, members, T, 8, 2, 16, nb)
    monkeypatch.setenv("SPECVERIFY_IDLE_NS", "5000000")
    for _ in range(3):
        err = h.i32([0])
        monkeypatch.setenv("SPECVERIFY_STALL_ROW", str(int(members[starts[1]])))
        _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == sv.SPEC_DERR_TIMEOUT
        monkeypatch.delenv("SPECVERIFY_STALL_ROW")
        err = h.i32([0])
        out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == 0
        check(out, q, pool, scales, bt, L)


@pytest.mark.parametrize("T,G,H,D,groups,forks,tiles,shared", [
    # measured row by row and shared, us
    (1, 8, 1, 128, 1, 32, 256, False),    # 46, 131: one item cut over all CTAs
    (1, 8, 1, 128, 2, 16, 256, False),    # 48, 84
    (1, 8, 1, 128, 1, 256, 24, False),    # 42, 55
    (1, 4, 8, 128, 1, 64, 12, False),     # 41, 54
    (5, 4, 1, 128, 1, 32, 256, False),    # 54, 73
    (5, 4, 8, 128, 8, 16, 8, False),      # 76, 93
    (5, 4, 8, 128, 8, 16, 16, False),     # 101, 107
    (5, 4, 8, 128, 8, 16, 32, True),      # 163, 148
    (5, 4, 8, 128, 1, 16, 32, False),     # 40, 52
    (5, 4, 8, 128, 1, 16, 256, True),     # 146, 110
    (5, 4, 8, 128, 1, 256, 2, False),     # 92, 130
    (5, 4, 8, 128, 1, 256, 24, True),     # 240, 179
    (16, 8, 8, 128, 8, 2, 8, False),      # 54, 72
    (16, 8, 8, 128, 8, 2, 64, True),      # 164, 137
    (8, 8, 8, 64, 2, 128, 32, True),      # 571, 371
])
def test_what_pays(monkeypatch, T, G, H, D, groups, forks, tiles, shared):
    """On both sides of where sharing pays: outputs with the bytes of kv_q8_attention's where it
    does not."""
    monkeypatch.delenv("SPECVERIFY_SHARE")
    rng = np.random.default_rng(30)
    L, bt, starts, members, nb = grouped(rng, [(128 * tiles, forks)] * groups, (10, 300), 0, 16, T)
    g = torch.Generator(device="cuda").manual_seed(30)
    shape = (nb, 1, 2, H)
    pool = (torch.randn((*shape, 16, D), device="cuda", generator=g) * 64).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(-7, -4, shape, device="cuda", generator=g).float())
    q = torch.randn((len(L), T, H * G, D), device="cuda", generator=g).bfloat16()
    args = q, pool, scales, h.i32(bt), h.i32(L)
    out, rows = torch.empty_like(q), torch.empty_like(q)
    sv.kv_q8_prefix_attention(*args, plan_of(bt, L, starts, members, T, G * H, H, 16, nb), out)
    sv.kv_q8_attention(*args, rows)
    assert torch.equal(out, rows) != shared


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_no_numbers(D, plain):
    """A NaN code among the shared values: that number of the outputs is NaN, as from
    kv_q8_attention, whatever the tile's scales are; the other codes of its tile are as ever."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(23, D=D)
    if not plain:
        scales[:, 0, 1] *= 1.5
    a, b = members[0], members[3]
    pool[bt[a, 2], 0, 1, 0, 5, 17] = 0x7f
    pool[bt[a, 3], 0, 1, 1, 0, D - 1] = 0xff
    pool[bt[b, 1], 0, 1, 1, 15, 0] = 0xff
    out = _run(dq, pool, scales, bt, L, plan_of(bt, L, starts, members, 4, 8, 2, 16, nb))
    want, spread, reach = q8.attention(q, pool, scales, bt, L)
    got, nan = out.double().cpu().numpy(), np.isnan(want)
    assert nan.any() and np.array_equal(np.isnan(got), nan)
    # code * scale is rounded to bf16 where the scale is no power of two: once more 2^-8
    lim = bound(want, spread, reach, D) + (0 if plain else 2.0 ** -8 * spread)
    assert (np.abs(got - want) <= lim)[~nan].all()
    rows = torch.empty_like(dq)
    sv.kv_q8_attention(dq, h.dev_pool(pool), h.dev_scales(scales), h.i32(bt), h.i32(L), rows)
    assert np.array_equal(torch.isnan(rows).cpu().numpy(), nan)


def test_the_largest_lists():
    """8192 rows in pairs, each pair with a tile in common, and one group of them all."""
    rng = np.random.default_rng(24)
    L, bt, starts, members, nb = grouped(rng, [(128, 2)] * 4096, (0, 20), 0, 16, 1)
    pool, scales = h.cache(rng, nb, 1, 1, 16, 64, spread=1)
    q, dq = queries(rng, len(L), 1, 2, 64)
    some = rng.permutation(len(L))[:200]
    for st in (starts, [0, len(L)]):
        err = h.i32([0])
        plan = plan_of(bt, L, st, members, 1, 2, 1, 16, nb, err=err)
        out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == 0
        check(out[torch.from_numpy(some).cuda()], q[some], pool, scales, bt[some], L[some])


def test_tables_wider_than_their_rows():
    """Entries that no row reaches change nothing, in whichever chunks of the tables they lie."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(25, groups=((9000, 3), (300, 2)))
    want = _run(dq, pool, scales, bt, L, plan_of(bt, L, starts, members, 4, 8, 2, 16, nb))
    check(want, q, pool, scales, bt, L)
    for more, fill in ((1, -1), (255, nb + 9), (70000, -1)):
        wide = np.concatenate([bt, np.full((len(L), more), fill)], 1)
        out = _run(dq, pool, scales, wide, L, plan_of(wide, L, starts, members, 4, 8, 2, 16, nb))
        assert torch.equal(out, want)
