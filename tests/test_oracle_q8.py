"""Pins of the 8-bit cache oracle and the block operators' oracle (CPU)."""
import numpy as np
import pytest

from oracle import pages, q8


def test_codes_match_the_format():
    import torch
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(q8.VALUES))
    fine = ~np.isnan(got)
    assert np.array_equal(got[fine], q8.VALUES[fine])
    x = np.concatenate([np.random.default_rng(1).normal(0, 30, 20000).astype(np.float32),
                        [0.0, -0.0, 2 ** -10, 3 * 2 ** -10, 17.0, 19.0, 448.0, -448.0]])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q8.encode(x.astype(np.float32)), want)


def test_block_scale_is_the_smallest_power_of_two():
    for a in (1e-30, 0.5, 1.0, 447.9, 448.0, 448.1, 3.3e38):
        s = q8.block_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -100 or a > 224 * s)
    assert q8.block_scale(0.0) == 2.0 ** -100


def test_append_by_hand():
    """Two tokens into a block that holds one: the old code moves to the coarser scale."""
    pool = np.zeros((2, 1, 2, 1, 4, 2), np.uint8)
    scales = np.ones((2, 1, 2, 1))
    pool[1, 0, 0, 0, 0] = q8.encode([1.0, -3.0])
    k = np.array([[[[900.0, 2.0]], [[0.5, -7.0]]]])
    p, s, err = q8.append(k, k, pool, scales, np.array([[1]]), [1])
    assert err == 0 and s[1, 0, 0, 0] == 4.0          # 900 / 4 = 225 <= 448 < 900 / 2 + 0
    got = q8.VALUES[p[1, 0, 0, 0]] * 4.0
    assert np.array_equal(got[0], [1.0, -3.0])        # exact: above the subnormals
    assert got[1, 0] == 896.0 and got[1, 1] == 2.0    # 225 -> 224
    assert np.array_equal(got[2], [0.5, -7.0])
    again = q8.append(k, k, p, s, np.array([[1]]), [1])
    assert np.array_equal(again[0], p) and np.array_equal(again[1], s)


def test_attention_by_hand():
    """One head, two keys, known weights; window and sinks; a query that sees nothing."""
    pool = np.zeros((1, 1, 2, 1, 4, 16), np.uint8)
    pool[0, 0, 0, 0, 1, 0] = q8.encode([1.0])[0]
    pool[0, 0, 1, 0, :3, 0] = q8.encode([1.0, 5.0, 9.0])
    q = np.zeros((1, 2, 1, 16))
    q[0, :, 0, 0] = np.log(3.0)
    args = (q, pool, np.ones((1, 1, 2, 1)), np.array([[0]]), [1])
    out, _, _ = q8.attention(*args, softmax_scale=1.0)
    assert np.isclose(out[0, 0, 0, 0], (1 + 3 * 5) / 4)
    assert np.isclose(out[0, 1, 0, 0], (1 + 3 * 5 + 9) / 5)
    out, _, _ = q8.attention(*args, softmax_scale=1.0, window=1)
    assert out[0, 0, 0, 0] == 5.0 and out[0, 1, 0, 0] == 9.0
    out, _, _ = q8.attention(*args, softmax_scale=1.0, window=1, sinks=1)
    assert np.isclose(out[0, 1, 0, 0], (1 + 9) / 2)
    out, _, _ = q8.attention(q, pool, np.ones((1, 1, 2, 1)), np.array([[0]]), [0],
                             softmax_scale=1.0, tree_mask=[[0, 2]])
    assert np.all(out[0, 0] == 0) and out[0, 1, 0, 0] == 5.0


def test_pages_by_hand():
    bt = np.array([[3, 1, -1], [-1, -1, -1], [-1, -1, -1]])
    sl, refs = np.array([5, 0, 0]), np.zeros(6, int)
    fs, ft = np.array([0, 2, 4, 5, -1, -1]), 4
    r = pages.reserve(bt, sl, fs, ft, 4, block_size=4, num_blocks=6)
    assert r["err"] == 0 and r["block_table"].tolist() == [[3, 1, 5], [4, -1, -1], [2, -1, -1]]
    assert r["free_top"] == 1
    f = pages.fork(bt, sl, refs, [0, 0], [2, 1], fs, ft, block_size=4, num_blocks=6)
    assert f["block_table"].tolist() == [[3, 1, -1], [3, 4, -1], [3, 5, -1]]
    assert f["extra_refs"].tolist() == [0, 0, 0, 2, 0, 0] and f["seq_lens"].tolist() == [5, 5, 5]
    assert f["copies"] == [(1, 5, 1), (1, 4, 1)] and f["free_top"] == 2
    g = pages.free(f["block_table"], f["seq_lens"], f["extra_refs"], [2, 0], fs, 2, num_blocks=6)
    assert g["err"] == 0 and g["extra_refs"].tolist() == [0] * 6
    assert g["free_stack"][:4].tolist() == [0, 2, 5, 1] and g["seq_lens"].tolist() == [0, 5, 0]
    h = pages.free(g["block_table"], g["seq_lens"], g["extra_refs"], [1], g["free_stack"], 4,
                   num_blocks=6)
    assert sorted(h["free_stack"].tolist()) == [0, 1, 2, 3, 4, 5] and h["free_top"] == 6
    bad = pages.fork(bt, sl, refs, [0, 1], [1, 2], fs, ft, block_size=4, num_blocks=6)
    assert bad["err"] == pages.BAD_SLOT and np.array_equal(bad["block_table"], bt)
    two = np.array([[3, -1], [3, -1]])
    assert pages.free(two, [1, 1], refs, [0, 1], fs, 2, num_blocks=6)["err"] == pages.BAD_BLOCK


@pytest.mark.parametrize("size,least,most", [(1, 0.0, 0.0), (64, 0.0, 3e-5), (512, 5e-5, 5e-4),
                                             (8192, 0.005, 0.03), (65536, 0.05, 0.3)])
def test_rejected_token_leaves_its_scale(size, least, most):
    """15 kept tokens of N(0, 1), a provisional one with a number of `size`, then the row's next
    token in its place: the scale stays, and the kept codes stay as that scale rounds them."""
    rng = np.random.default_rng(9)
    kept, draft, new = (rng.normal(0, 1, (1, n, 1, 128)) for n in (15, 1, 1))
    draft[0, 0, 0, 5] = size
    bt, at = np.array([[0]]), np.array([15])
    pool, scales = np.zeros((1, 1, 2, 1, 16, 128), np.uint8), np.zeros((1, 1, 2, 1))
    pool, scales, _ = q8.append(kept, kept, pool, scales, bt, np.array([0]))
    drafted = q8.append(draft, draft, pool, scales, bt, at)
    after = q8.append(new, new, drafted[0], drafted[1], bt, at)
    plain = q8.append(new, new, pool, scales, bt, at)
    values = [q8.VALUES[x[0][0, 0, 0, 0, :15]] * x[1][0, 0, 0, 0] for x in (after, plain)]
    assert np.array_equal(after[1], drafted[1])
    change = np.linalg.norm(values[0] - values[1]) / np.linalg.norm(values[1])
    assert least <= change <= most


@pytest.mark.parametrize("bs", [1, 4, 16])
def test_fork_and_free_leak_nothing(bs):
    """Random forks and frees: every block always has extra_refs + 1 holders or lies on the stack."""
    rng = np.random.default_rng(bs)
    B, MB, nb = 12, 6, 60
    s = dict(block_table=np.full((B, MB), -1), seq_lens=np.zeros(B, int),
             extra_refs=np.zeros(nb, int), free_stack=rng.permutation(nb), free_top=np.array(nb))
    for _ in range(200):
        rows = np.nonzero(s["seq_lens"] == 0)[0]
        live = np.nonzero(s["seq_lens"])[0]
        kind = rng.integers(3)
        if kind == 0 and len(rows):
            n = np.zeros(B, int)
            n[rng.choice(rows)] = rng.integers(1, MB * bs + 1)
            r = pages.reserve(s["block_table"], s["seq_lens"], s["free_stack"], s["free_top"], 0,
                              block_size=bs, num_blocks=nb, num_new=n)
            if r["err"] == 0:
                s["seq_lens"] = s["seq_lens"] + n
        elif kind == 1 and len(live) and len(rows) > 1:
            dst = rng.choice(rows, 2, replace=False)
            r = pages.fork(s["block_table"], s["seq_lens"], s["extra_refs"],
                           rng.choice(live, 2), dst, s["free_stack"], s["free_top"],
                           block_size=bs, num_blocks=nb)
        elif kind == 2 and len(live):
            pick = rng.choice(live, rng.integers(1, len(live) + 1), replace=False)
            r = pages.free(s["block_table"], s["seq_lens"], s["extra_refs"], pick,
                           s["free_stack"], s["free_top"], num_blocks=nb)
            assert r["err"] == 0
        else:
            continue
        s.update({k: v for k, v in r.items() if k in s})
        held = np.bincount(s["block_table"][s["block_table"] >= 0], minlength=nb)
        stack = np.bincount(s["free_stack"][:int(s["free_top"])], minlength=nb)
        assert np.all((held > 0) + stack == 1)
        assert np.array_equal(s["extra_refs"], np.maximum(held - 1, 0))
