"""kv_q8_append and kv_q8_attention against the fp64 oracle."""
import numpy as np
import pytest

from gpu_helpers import gpu_lib
from oracle import q8
from q8_helpers import (as_int32, bf16_values, cache, dev_pool, dev_scales, i32, poison_tails,
                        table, tree_masks)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
def _append_case(seed, *, lengths, T, H, D, bs, dtype, num_new=None, layers=2, layer=1):
    import torch
    rng = np.random.default_rng(seed)
    B = len(lengths)
    n = [T] * B if num_new is None else num_new
    bt, _, nb = table(rng, [a + b for a, b in zip(lengths, n)], bs)
    pool, scales = cache(rng, nb, layers, H, bs, D)
    # magnitudes over several binades, so that some blocks' scales grow and some do not
    k, v = (rng.normal(0, 1, (B, T, H, D)) * 2.0 ** rng.integers(-6, 7, (B, T, H, 1))
            for _ in range(2))
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v = (torch.from_numpy(x.astype(np.float32)).to(t) for x in (k, v))
    return dict(k=k, v=v, pool=pool, scales=scales, bt=bt, sl=np.array(lengths),
                nn=None if num_new is None else np.array(num_new), layer=layer)


def _append_gpu(sv, c, stream=None):
    import torch
    pool, scales = dev_pool(c["pool"]), dev_scales(c["scales"])
    err = i32([0])
    sv.kv_q8_append(c["k"].cuda(), c["v"].cuda(), pool, scales, i32(c["bt"]), i32(c["sl"]),
                    layer=c["layer"], num_new=None if c["nn"] is None else i32(c["nn"]),
                    err_flag=err)
    torch.cuda.synchronize()
    return pool.view(torch.uint8).cpu().numpy(), scales.double().cpu().numpy(), int(err.item())


def _append_same(sv, c):
    want = q8.append(c["k"].double().numpy(), c["v"].double().numpy(), c["pool"], c["scales"],
                     c["bt"], c["sl"], c["nn"], layer=c["layer"])
    got = _append_gpu(sv, c)
    assert got[2] == want[2]
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])
    return want


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,D,bs", [(1, 2, 128, 16), (5, 8, 128, 16), (3, 1, 64, 32),
                                      (70, 2, 64, 16), (40, 3, 256, 64), (9, 2, 80, 1),
                                      (17, 1, 16, 24), (200, 1, 128, 128)])
def test_append_matches_oracle(dtype, T, H, D, bs):
    lengths = [0, 1, bs - 1, bs, bs + 1, 3 * bs + bs // 2, 7]
    _append_same(gpu_lib(), _append_case(T * bs, lengths=lengths, T=T, H=H, D=D, bs=bs,
                                         dtype=dtype))


def test_append_ragged_and_empty_rows():
    c = _append_case(3, lengths=[0, 5, 16, 31, 100], T=33, H=2, D=128, bs=16, dtype="bf16",
                     num_new=[0, 33, 1, 0, 17])
    _append_same(gpu_lib(), c)


def test_append_zeros_extremes_and_subnormals():
    import torch
    c = _append_case(4, lengths=[0, 3, 16], T=4, H=2, D=64, bs=16, dtype="fp32")
    c["k"][0] = 0
    c["k"][1, :, 0] *= 1e-44      # below the smallest scale
    c["k"][1, :, 1] = 3.3e38
    c["v"][2, 0, 0, 0] = 448.0
    c["v"][2, 0, 1] = torch.linspace(-1, 1, 64) * 2.0 ** -120
    _append_same(gpu_lib(), c)


def test_append_reports_what_it_cannot_store():
    sv = gpu_lib()
    c = _append_case(5, lengths=[2, 20, 0], T=5, H=2, D=64, bs=16, dtype="bf16")
    c["k"][0, 1, 0, 3] = float("nan")
    c["v"][1, 2, 1, 7] = float("inf")
    c["v"][2, 0, 0, 0] = -float("inf")
    assert _append_same(sv, c)[2] == 256
    c = _append_case(6, lengths=[2, 20, 0, 6, 7], T=5, H=2, D=64, bs=16, dtype="bf16",
                     num_new=[5, 5, 5, 6, 5])
    c["bt"][1, 1] = len(c["pool"])
    c["bt"][4, 0] = -1
    c["sl"][2] = -1
    assert _append_same(sv, c)[2] == 32 | 8
    c = _append_case(7, lengths=[40], T=5, H=1, D=64, bs=16, dtype="bf16")
    c["sl"][0] = 44   # 49 tokens in 3 blocks of 16
    assert _append_same(sv, c)[2] == 8


def test_append_twice_changes_nothing():
    sv = gpu_lib()
    c = _append_case(8, lengths=[3, 18], T=6, H=2, D=128, bs=16, dtype="bf16")
    pool, scales, _ = _append_gpu(sv, c)
    c2 = dict(c, pool=pool, scales=scales)
    again = _append_gpu(sv, c2)
    assert np.array_equal(again[0], pool) and np.array_equal(again[1], scales)


# ------------------------------------------------------------------ attention
def _attn_case(seed, *, lengths, T, Hq, H, D, bs, num_new=None, tree=False, dtype="bf16", layers=2,
               layer=1, qscale=1.0, spread=1):
    rng = np.random.default_rng(seed)
    B = len(lengths)
    n = [T] * B if num_new is None else num_new
    ends = [a + b for a, b in zip(lengths, n)]
    bt, _, nb = table(rng, ends, bs)
    pool, scales = cache(rng, nb, layers, H, bs, D, spread)
    pool = poison_tails(pool, bt, ends, bs)
    q = rng.normal(0, qscale, (B, T, Hq, D))
    q = bf16_values(q) if dtype == "bf16" else q.astype(np.float32).astype(np.float64)
    return dict(q=q, pool=pool, scales=scales, bt=bt, sl=np.array(lengths),
                nn=None if num_new is None else np.array(num_new), layer=layer, dtype=dtype,
                tree=tree_masks(rng, B, T) if tree else None)


def _attn_gpu(sv, c, **kw):
    import torch
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    q = torch.from_numpy(c["q"]).to(dt).cuda()
    out = torch.full_like(q, 7.0)
    err = i32([0])
    sv.kv_q8_attention(q, dev_pool(c["pool"]), dev_scales(c["scales"]), i32(c["bt"]), i32(c["sl"]),
                       out, layer=c["layer"], num_new=None if c["nn"] is None else i32(c["nn"]),
                       tree_mask=None if c["tree"] is None else i32(as_int32(c["tree"])),
                       err_flag=err, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), int(err.item())


def _bound(c, want, spread, reach, D):
    """What the arithmetic may be off by.

    A score carries D fp32 products and sums (2^-24 each relative to sum |q_d k_d|, `reach`),
    counted 16-fold for the accumulation order and width of the matrix units, and an fp32
    exponential: the weight's relative error is e = 16 D 2^-24 reach + 2^-20, in the weight and
    in the sum. bf16: a weight is held in 9 bits (2^-9 of it; 2^-16 of the largest for the
    smallest ones) and the output rounded to 8 (2^-8 of it). fp32: 2^-24, and fp32 sums.
    """
    e = 2 * (16 * D * 2.0 ** -24 * reach + 2.0 ** -20)
    n = c["bt"].shape[1] * c["pool"].shape[4]
    if c["dtype"] == "bf16":
        return (2.0 ** -9 + e) * spread + 2.0 ** -8 * np.abs(want) + n * 2.0 ** -22 * spread + 1e-30
    return (e + 64 * 2.0 ** -24) * spread + 2.0 ** -23 * np.abs(want) + 1e-30


def _attn_same(sv, c, kw=None, oracle_kw=None):
    kw = kw or {}
    got, err = _attn_gpu(sv, c, **kw)
    want, spread, reach = q8.attention(c["q"], c["pool"], c["scales"], c["bt"], c["sl"], c["nn"],
                                       layer=c["layer"], tree_mask=c["tree"], **kw)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    off = np.abs(got - want)[ok]
    lim = _bound(c, want, spread, reach, c["q"].shape[-1])[ok]
    worst = float(np.max(off / lim)) if off.size else 0.0
    assert worst <= 1.0, worst
    return err


LENGTHS = [0, 1, 15, 16, 123, 127, 128, 129, 300]


@pytest.mark.parametrize("T,Hq,H,D,bs", [
    (1, 4, 1, 128, 16), (5, 8, 2, 128, 16), (1, 1, 1, 128, 16), (3, 12, 4, 128, 32),
    (7, 8, 1, 128, 64), (32, 4, 1, 128, 16), (16, 16, 2, 128, 128), (2, 7, 1, 128, 8),
    (5, 8, 2, 64, 16), (1, 8, 1, 64, 32), (32, 12, 1, 64, 64), (4, 2, 1, 128, 256),
    (1, 2, 1, 80, 16), (5, 4, 2, 256, 16), (3, 2, 2, 16, 24), (2, 2, 1, 128, 1),
])
def test_attention_matches_oracle(T, Hq, H, D, bs):
    c = _attn_case(T * D + bs, lengths=LENGTHS, T=T, Hq=Hq, H=H, D=D, bs=bs)
    assert _attn_same(gpu_lib(), c) == 0


@pytest.mark.parametrize("T,G,D,bs", [(1, 2, 128, 16), (5, 4, 128, 16), (5, 4, 64, 32),
                                      (7, 4, 128, 64), (12, 4, 128, 16), (16, 4, 128, 16),
                                      (16, 4, 64, 16)])
def test_attention_many_items_a_cta(T, G, D, bs):
    """1200 (row, kv head) pairs of one to three tiles: every CTA goes through several, so that
    what it keeps of an item is used again, for each number of query rows."""
    rng = np.random.default_rng(T * G + D)
    c = _attn_case(T * G + D, lengths=[int(x) for x in rng.integers(0, 300, 150)], T=T, Hq=8 * G,
                   H=8, D=D, bs=bs)
    assert _attn_same(gpu_lib(), c) == 0


@pytest.mark.parametrize("T,Hq,H,D,bs", [(1, 4, 1, 128, 16), (5, 4, 2, 64, 16), (9, 3, 1, 48, 5)])
def test_attention_fp32(T, Hq, H, D, bs):
    c = _attn_case(T * D + bs, lengths=LENGTHS, T=T, Hq=Hq, H=H, D=D, bs=bs, dtype="fp32")
    assert _attn_same(gpu_lib(), c) == 0


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32), (96, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (37, 4), (128, 0), (129, 200), (250, 37),
                                          (5000, 3)])
def test_attention_window_and_sinks(D, bs, window, sinks):
    c = _attn_case(window + D, lengths=[0, 1, 60, 129, 401, 700, 1023], T=6, Hq=4, H=1, D=D, bs=bs)
    assert _attn_same(gpu_lib(), c, dict(window=window, sinks=sinks)) == 0


NO_LIMIT = 2 ** 31 - 1


@pytest.mark.parametrize("T,G,D,bs,dtype", [(6, 4, 128, 16, "bf16"), (32, 2, 64, 32, "bf16"),
                                            (6, 4, 96, 16, "bf16"), (3, 2, 128, 16, "fp32")])
@pytest.mark.parametrize("window,sinks", [(NO_LIMIT, 0), (NO_LIMIT, NO_LIMIT), (NO_LIMIT - 20, 4),
                                          (1, NO_LIMIT), (2 ** 30, 1)])
def test_attention_largest_windows(T, G, D, bs, dtype, window, sinks):
    """Windows and sinks that stand for "no limit": arithmetic on them must not leave 32 bits."""
    c = _attn_case(D + T, lengths=[0, 1, 60, 127, 300], T=T, Hq=2 * G, H=2, D=D, bs=bs, dtype=dtype)
    assert _attn_same(gpu_lib(), c, dict(window=window, sinks=sinks)) == 0


@pytest.mark.parametrize("T,G,D,bs", [(15, 4, 128, 16), (32, 2, 128, 64), (9, 1, 64, 16),
                                      (5, 2, 32, 16)])
def test_attention_tree(T, G, D, bs):
    c = _attn_case(T, lengths=[0, 3, 120, 128, 250], T=T, Hq=2 * G, H=2, D=D, bs=bs, tree=True)
    assert _attn_same(gpu_lib(), c) == 0
    c["tree"][:, 1] = 0   # with no committed token: a query that sees nothing
    assert _attn_same(gpu_lib(), c) == 0


def test_attention_ragged_rows():
    c = _attn_case(11, lengths=[0, 40, 128, 0, 77], T=6, Hq=8, H=2, D=128, bs=16,
                   num_new=[0, 6, 1, 3, 0])
    assert _attn_same(gpu_lib(), c) == 0


def test_attention_many_rows_and_splits():
    """More items than CTAs, lengths from one token to thousands: items that begin and end
    anywhere in a CTA's share."""
    rng = np.random.default_rng(12)
    lengths = [int(x) for x in rng.integers(0, 200, 150)] + [2500, 0, 1]
    c = _attn_case(12, lengths=lengths, T=2, Hq=8, H=4, D=128, bs=16, layers=1, layer=0)
    assert _attn_same(gpu_lib(), c) == 0


def test_attention_long_row():
    c = _attn_case(13, lengths=[20000], T=3, Hq=2, H=1, D=128, bs=16, layers=1, layer=0)
    assert _attn_same(gpu_lib(), c) == 0
    c = _attn_case(14, lengths=[20000, 17], T=2, Hq=8, H=1, D=64, bs=64, layers=1, layer=0)
    assert _attn_same(gpu_lib(), c) == 0


@pytest.mark.parametrize("D", [128, 64, 96])
def test_attention_peaked_scores(D):
    """Scores over hundreds of binades: later keys far above the first tiles' maximum and far
    below it, scales that differ by 2^24 from block to block."""
    c = _attn_case(15 + D, lengths=[600, 900], T=4, Hq=4, H=1, D=D, bs=16, qscale=6.0, spread=12)
    c["scales"][:, :, 0] = np.minimum(c["scales"][:, :, 0], 2.0 ** -3)
    # the row's keys grow along the sequence
    for b in range(2):
        held = c["bt"][b][c["bt"][b] >= 0]
        c["scales"][held, :, 0] = 2.0 ** np.linspace(-12, -3, len(held)).round()[:, None, None]
    assert _attn_same(gpu_lib(), c) == 0


@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (5, 4, 64), (16, 4, 128)])
@pytest.mark.parametrize("first,rest", [(-100, 4), (-100, 60), (-100, 110), (-100, 0), (60, -60),
                                        (-60, 60), (0, -100), (110, -100), (-100, -100), (110, 110), (-90, -90)])
def test_attention_value_scales_far_apart(T, G, D, first, rest):
    """V scales of the first tile 2^first (2^-100: its values were zero), of the others 2^rest, of
    every fifth block in between; 1200 rows over the same two rows' blocks, so that a CTA takes
    whole rows."""
    c = _attn_case(24 + T, lengths=[150, 1000], T=T, Hq=G, H=1, D=D, bs=16)
    for row in c["bt"]:
        for j, x in enumerate(row[row >= 0]):
            e = first if j < 8 else (first + rest) // 2 if j % 5 == 0 else rest
            c["scales"][x, :, 1] = 2.0 ** e
            if e == -100:
                c["pool"][x, :, 1] &= 0x80
    many = dict(c, **{k: np.tile(c[k], (600,) + (1,) * (c[k].ndim - 1)) for k in ("q", "bt", "sl")})
    got, err = _attn_gpu(gpu_lib(), many)
    want, spread, reach = q8.attention(c["q"], c["pool"], c["scales"], c["bt"], c["sl"], layer=1)
    lim = _bound(c, want, spread, reach, D)
    got = got.reshape(600, *want.shape)
    assert err == 0 and np.isfinite(got).all()
    assert np.max(np.abs(got - want) / lim) <= 1.0


def _tail_bound(want, spread, codes2, top):
    """bf16 output, half a step: 2^-8. A weight is held in 9 bits (half a step 2^-9), and q . k is
    exact here; a score in log2 units is below 64, rounded to 2^-19 twice, in the weight and in the
    sum, whose exponentials and additions are fp32: 2^-16. A small weight is cut to one of the two
    multiples of a step next to it, by turns: off by half a step in the mean square, so the sum
    over the keys by less than 8 times step / 2 * sqrt(sum of squared codes). The step is 2^-24 of
    the row's reference, which is at most twice the largest product of weight and V scale."""
    return (2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -16) * spread
            + 8 * 2.0 ** -24 * top * np.sqrt(codes2))


@pytest.mark.parametrize("G", [4, 20, 40, 64])
@pytest.mark.parametrize("low,high,sign", [(2.75, 5.5, 1), (2.75, 5.5, -1), (-0.5, 3.0, 1),
                                           (0.0, 0.0, 1)])
def test_attention_many_small_probabilities(G, low, high, sign):
    """One key with most of the weight and V = 0, then 100 thousand with 2^-18 to 2^-27 of its
    probability each and V of one sign: what the small ones lose adds up. About as many rows as
    there are CTAs share the blocks, so that a row lies in one CTA or two."""
    import torch
    sv = gpu_lib()
    rng = np.random.default_rng(G)
    N, bs, D = 100 * 1024, 64, 64
    rows = 300
    nb = N // bs
    pool = np.zeros((nb, 1, 2, 1, bs, D), np.uint8)
    grid = q8.VALUES[:127]
    grid = np.concatenate([-grid[1:], grid])
    k = rng.choice(grid[(grid >= low) & (grid <= high)], N)
    k[0] = 18.0
    v = rng.integers(64, 448, (N, D)).astype(np.float64)
    v[0] = 0.0
    pool[:, 0, 0, 0, :, 0] = q8.encode(k).reshape(nb, bs)
    pool[:, 0, 1, 0] = q8.encode(sign * v).reshape(nb, bs, D)
    v = q8.VALUES[pool[:, 0, 1, 0]].reshape(N, D)
    scales = np.ones((nb, 1, 2, 1))
    scales[:, 0, 1] = 2.0 ** -8
    q = np.zeros((rows, 1, G, D))
    q[..., 0] = rng.choice([1.0, 0.984375, 1.015625], (rows, 1, G))   # bf16 numbers
    bt = np.tile(np.append(0, 1 + rng.permutation(nb - 1)), (rows, 1))
    k, v = (x.reshape(nb, bs, -1)[bt[0]].reshape(N, -1) for x in (k, v))
    x = torch.from_numpy(q).bfloat16().cuda()
    out = torch.empty_like(x)
    sv.kv_q8_attention(x, dev_pool(pool), dev_scales(scales), i32(bt), i32([N - 1] * rows), out,
                       softmax_scale=1.0)
    got = out.double().cpu().numpy()
    for f in (1.0, 0.984375, 1.015625):
        z = f * k[:, 0]
        w = np.exp(z - z.max())
        w /= w.sum()
        want = w @ v * 2.0 ** -8
        lim = _tail_bound(want, w @ np.abs(v) * 2.0 ** -8, (v * v).sum(0), w.max() * 2.0 ** -8)
        off = np.abs(got[q[..., 0] == f] - want)
        assert off.size and np.max(off / lim) <= 1.0, float(np.max(off / lim))


def test_attention_softmax_scale_and_small_queries():
    sv = gpu_lib()
    c = _attn_case(16, lengths=[200, 50], T=2, Hq=4, H=1, D=128, bs=16)
    assert _attn_same(sv, c, dict(softmax_scale=0.5)) == 0
    c["q"] *= 2.0 ** -40
    c["q"][0, 0, 0] = 0.0
    c["q"][1, 1, 2, 5:] *= 2.0 ** -30   # numbers far below their row's largest
    assert _attn_same(sv, c) == 0


@pytest.mark.parametrize("D,T", [(128, 1), (64, 5), (128, 16)])
@pytest.mark.parametrize("largest", [1.0, 1.9921875])
@pytest.mark.parametrize("e", [-3, -8, -9, -10, -11, -14])
def test_attention_small_query_numbers(D, T, largest, e):
    """Numbers down to 2^-9 of their row's largest are exact, smaller ones are off by up to 2^-17
    of it. The score, 2, is the difference of two products of 256."""
    import torch
    sv = gpu_lib()
    y = 2.0 ** e
    x = y * (1 + 2.0 ** -7)
    q = np.zeros((1, T, 4, D))
    q[..., 0], q[..., 1], q[..., 2] = largest, x, y
    pool = np.zeros((1, 1, 2, 1, 64, D), np.uint8)
    pool[0, 0, 0, 0, 1, 1:3] = q8.encode(np.array([256.0, -256.0]))
    pool[0, 0, 1, 0, 1] = q8.encode(256.0)
    scales = np.ones((1, 1, 2, 1))
    scales[0, 0, 0] = 2.0 ** -e
    out = torch.empty((1, T, 4, D), dtype=torch.bfloat16, device="cuda")
    sv.kv_q8_attention(torch.from_numpy(q).bfloat16().cuda(), dev_pool(pool), dev_scales(scales),
                       i32([[0]]), i32([1]), out, softmax_scale=1.0, num_new=i32([1]))
    got = out.double().cpu().numpy()[0, 0]
    # keys of scores 0 and 2, values 0 and 256
    off = 0.0 if y >= 2.0 ** -9 * largest else 2 * 256 * 2.0 ** -e * largest * 2.0 ** -17
    lo, hi = (256 / (1 + np.exp(-(2 + d))) for d in (-off, off))
    tol = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -16
    assert np.all(got >= lo * (1 - tol)) and np.all(got <= hi * (1 + tol))


def test_attention_zero_scales():
    c = _attn_case(17, lengths=[200, 50], T=2, Hq=4, H=1, D=128, bs=16)
    c["scales"][:, :, 1] = 0.0
    assert _attn_same(gpu_lib(), c) == 0
    c["scales"][:, :, 0] = 2.0 ** -100
    assert _attn_same(gpu_lib(), c) == 0


@pytest.mark.parametrize("D", [128, 96])
def test_attention_nan_queries_stay_in_their_row(D):
    c = _attn_case(18, lengths=[140, 50], T=3, Hq=4, H=1, D=D, bs=16)
    c["q"][0, 1, 2, 7] = np.nan
    got, err = _attn_gpu(gpu_lib(), c)
    c["q"][0, 1, 2, 7] = 0.0
    want, spread, reach = q8.attention(c["q"], c["pool"], c["scales"], c["bt"], c["sl"], None,
                                       layer=c["layer"])
    bad = np.zeros(got.shape, bool)
    bad[0, 1, 2] = True
    assert err == 0 and np.array_equal(np.isnan(got), bad)
    assert np.all(np.abs(got - want)[~bad] <= _bound(c, want, spread, reach, D)[~bad])


@pytest.mark.parametrize("D", [128, 64, 96])
def test_attention_bad_blocks_and_lengths(D):
    sv = gpu_lib()
    c = _attn_case(19, lengths=[300, 300, 10, 60, 5], T=3, Hq=4, H=2, D=D, bs=16,
                   num_new=[3, 3, 3, 4, 3])
    c["bt"][0, 3] = -1
    c["bt"][1, 0] = len(c["pool"]) + 5
    c["sl"][2] = -4
    assert _attn_same(sv, c) == 32 | 8
    # a bad block outside every window is not touched
    c = _attn_case(20, lengths=[600, 600], T=3, Hq=4, H=2, D=D, bs=16)
    c["bt"][0, 10] = -1
    assert _attn_same(sv, c, dict(window=100, sinks=4)) == 0


def test_attention_runs_on_the_given_stream_and_repeats():
    """Two streams at once, each with the workspace of its own; the same bits every time."""
    import torch
    sv = gpu_lib()
    c = _attn_case(21, lengths=[3000, 700, 90], T=5, Hq=8, H=2, D=128, bs=16)
    q = torch.from_numpy(c["q"]).bfloat16().cuda()
    args = (dev_pool(c["pool"]), dev_scales(c["scales"]), i32(c["bt"]), i32(c["sl"]))
    first = torch.empty_like(q)
    sv.kv_q8_attention(q, *args, first, layer=1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(10)] for _ in streams]
    for i in range(10):
        for s, o in zip(streams, outs):
            sv.kv_q8_attention(q, *args, o[i], layer=1, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for x in o:
            assert torch.equal(x, first)


def test_append_then_attend_in_a_graph():
    """The pair captured once and replayed on new tokens and lengths."""
    import torch
    sv = gpu_lib()
    c = _attn_case(22, lengths=[40, 130], T=3, Hq=4, H=2, D=128, bs=16)
    rng = np.random.default_rng(22)
    q = torch.from_numpy(c["q"]).bfloat16().cuda()
    k, v = (torch.empty((2, 3, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool, scales = dev_pool(c["pool"]), dev_scales(c["scales"])
    bt, sl, out = i32(c["bt"]), i32(c["sl"]), torch.empty_like(q)

    def step():
        sv.kv_q8_append(k, v, pool, scales, bt, sl, layer=1)
        sv.kv_q8_attention(q, pool, scales, bt, sl, out, layer=1)

    k.zero_(), v.zero_()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for shift in (0, -7, -40):
        pool.copy_(dev_pool(c["pool"]))
        scales.copy_(dev_scales(c["scales"]))
        kv = [bf16_values(rng.normal(0, 1, (2, 3, 2, 128))) for _ in range(2)]
        k.copy_(torch.from_numpy(kv[0]).bfloat16())
        v.copy_(torch.from_numpy(kv[1]).bfloat16())
        L = c["sl"] + shift
        sl.copy_(i32(L))
        graph.replay()
        torch.cuda.synchronize()
        p2, s2, _ = q8.append(kv[0], kv[1], c["pool"], c["scales"], c["bt"], L, layer=1)
        assert np.array_equal(pool.view(torch.uint8).cpu().numpy(), p2)
        want, spread, reach = q8.attention(c["q"], p2, s2, c["bt"], L, layer=1)
        off = np.abs(out.double().cpu().numpy() - want)
        assert np.all(off <= _bound(c, want, spread, reach, 128))


def _attend(sv, c, out, stream=None):
    """A call on the case's device tensors, kept in the case."""
    import torch
    if "dev" not in c:
        c["dev"] = (torch.from_numpy(c["q"]).bfloat16().cuda(), dev_pool(c["pool"]),
                    dev_scales(c["scales"]), i32(c["bt"]), i32(c["sl"]))
    sv.kv_q8_attention(*c["dev"], out, layer=c["layer"], stream=stream)


def test_attention_graph_outlives_a_larger_workspace():
    """A graph of a small shape, then a larger shape on its stream and new tensors wherever there
    is memory: the replay neither uses nor changes what is not its own."""
    import torch
    sv = gpu_lib()
    small = _attn_case(25, lengths=[5000, 700], T=1, Hq=4, H=2, D=64, bs=16)
    large = _attn_case(26, lengths=[3000, 90], T=32, Hq=4, H=2, D=128, bs=16)
    assert (sv.kv_q8_attention_workspace_bytes(32, 4, 2, 128)
            > sv.kv_q8_attention_workspace_bytes(1, 4, 2, 64))
    s = torch.cuda.Stream()
    want, out = (torch.empty((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    big = torch.empty((2, 32, 4, 128), dtype=torch.bfloat16, device="cuda")
    _attend(sv, small, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        _attend(sv, small, out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        _attend(sv, small, out)
    with torch.cuda.stream(s):
        _attend(sv, large, big)
    torch.cuda.synchronize()
    sizes = [sv.kv_q8_attention_workspace_bytes(*x) + 256 for x in ((1, 4, 2, 64), (32, 4, 2, 128))]
    with torch.cuda.stream(s):
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in 3 * sizes]
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((x == 7).all()) for x in others)


def test_attention_graphs_of_one_stream_replayed_on_two():
    import torch
    sv = gpu_lib()
    s = torch.cuda.Stream()
    got = []
    for seed, lengths in ((27, [9000, 300]), (28, [100, 8000])):
        c = _attn_case(seed, lengths=lengths, T=4, Hq=8, H=2, D=128, bs=16)
        want, out = (torch.empty((2, 4, 8, 128), dtype=torch.bfloat16, device="cuda")
                     for _ in range(2))
        _attend(sv, c, want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            _attend(sv, c, out)
        got.append((graph, out, want, torch.cuda.Stream(), c))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, out, _, stream, _ in got:
            with torch.cuda.stream(stream):
                out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in got:
        assert torch.equal(out, want)


def test_attention_workspace_is_allocated_in_its_streams_order():
    """Memory that was just freed on the current stream may still be in use there: a call on
    another stream must not take it."""
    import torch
    sv = gpu_lib()
    c = _attn_case(29, lengths=[3000, 700], T=5, Hq=8, H=2, D=128, bs=16)
    out = torch.empty((2, 5, 8, 128), dtype=torch.bfloat16, device="cuda")
    n = sv.kv_q8_attention_workspace_bytes(5, 8, 2, 128) + 256
    _attend(sv, c, out)
    torch.cuda.synchronize()
    x = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    was = {t.data_ptr() for t in x}
    del x
    s = torch.cuda.Stream(priority=-1)
    _attend(sv, c, out, stream=s)
    held = sv._attn_workspaces[(out.device.index, s.cuda_stream)]
    assert held.data_ptr() not in was
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,G,D,rows,stall", [
    (5, 4, 128, 8, 3), (5, 4, 64, 8, 0), (12, 4, 128, 8, 7), (16, 4, 128, 8, 3), (8, 4, 128, 8, 0),
    (16, 4, 64, 8, 2), (1, 1, 128, 8, 2), (16, 4, 128, 160, 80), (12, 4, 128, 160, 5)])
def test_attention_wait_runs_out(monkeypatch, T, G, D, rows, stall):
    """SPECVERIFY_STALL_ROW withholds a row's V tiles: the waits of the CTAs that have it run out
    (after 5 ms instead of 2 s), the call ends and reports it, and the CTAs that work on other
    rows are not concerned. The next call is as ever."""
    import torch
    sv = gpu_lib()
    rng = np.random.default_rng(30)
    top = 3000 if rows < 100 else 700
    c = _attn_case(30, lengths=[int(x) for x in rng.integers(top // 2, top, rows)], T=T, Hq=8 * G,
                   H=8, D=D, bs=16, layers=1, layer=0)
    want, hurt, again = (torch.empty((rows, T, 8 * G, D), dtype=torch.bfloat16, device="cuda")
                         for _ in range(3))
    _attend(sv, c, want)
    err = i32([0])
    torch.cuda.synchronize()
    monkeypatch.setenv("SPECVERIFY_STALL_ROW", str(stall))
    monkeypatch.setenv("SPECVERIFY_IDLE_NS", "5000000")
    sv.kv_q8_attention(*c["dev"], hurt, layer=c["layer"], err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == sv.SPEC_DERR_TIMEOUT
    # a CTA has less than a row
    far = [b for b in range(rows) if abs(b - stall) > 1]
    assert torch.equal(hurt[far], want[far])
    monkeypatch.delenv("SPECVERIFY_STALL_ROW")
    monkeypatch.delenv("SPECVERIFY_IDLE_NS")
    err.zero_()
    sv.kv_q8_attention(*c["dev"], again, layer=c["layer"], err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(again, want)


def test_binding_refuses():
    import torch
    sv = gpu_lib()
    c = _attn_case(23, lengths=[20], T=2, Hq=4, H=2, D=64, bs=16)
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    pool, scales, bt, sl = dev_pool(c["pool"]), dev_scales(c["scales"]), i32(c["bt"]), i32(c["sl"])
    out = torch.empty_like(q)
    ok = dict(q=q, kv_pool=pool, kv_scales=scales, block_table=bt, seq_lens=sl, out=out)
    sv.kv_q8_attention(**ok)
    for err, change in [
        (TypeError, dict(q=q.half(), out=out.half())), (TypeError, dict(kv_pool=pool.to(torch.bfloat16))),
        (TypeError, dict(kv_scales=scales.double())), (ValueError, dict(kv_scales=scales[:-1])),
        (ValueError, dict(out=out[:, :1].contiguous())), (TypeError, dict(out=out.float())),
        (ValueError, dict(q=q.transpose(1, 2))), (ValueError, dict(seq_lens=i32([1, 2]))),
        (TypeError, dict(seq_lens=sl.long())), (ValueError, dict(block_table=bt.repeat(2, 1))),
        (ValueError, dict(tree_mask=i32([[1]]))), (ValueError, dict(num_new=i32([1, 1]))),
        (sv.SpecError, dict(layer=2)), (sv.SpecError, dict(sinks=3)),
        (sv.SpecError, dict(softmax_scale=0.0)),
        (sv.SpecError, dict(workspace=torch.empty(300, dtype=torch.uint8, device="cuda"))),
        (sv.SpecError, dict(q=q[:, :, :3].contiguous(), out=out[:, :, :3].contiguous())),
    ]:
        with pytest.raises(err):
            sv.kv_q8_attention(**{**ok, **change})
    kv = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    ok = dict(k=kv, v=kv, kv_pool=pool, kv_scales=scales, block_table=bt, seq_lens=sl)
    sv.kv_q8_append(**ok)
    for err, change in [(TypeError, dict(v=kv.float())), (ValueError, dict(v=kv[:, :1].contiguous())),
                        (TypeError, dict(k=kv.half(), v=kv.half())), (sv.SpecError, dict(layer=-1)),
                        (ValueError, dict(k=kv[..., :32].contiguous(), v=kv[..., :32].contiguous()))]:
        with pytest.raises(err):
            sv.kv_q8_append(**{**ok, **change})
    torch.cuda.synchronize()
