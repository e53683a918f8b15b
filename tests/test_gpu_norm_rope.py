"""Norms and rotary positions, with and without the 8-bit cache, against the fp64 oracle.

Error bound. With u = 2^-24: the sum of squares of a head is off by at most 21 u of itself (16
terms of a lane and 5 steps across lanes), its mean by 3 u more, so 1 / sqrt by 12 u and 4 u of its
own, a normed number by 18 u; cos and sin by 4 u (2 of the angle, 2 of the polynomial and the
factor), a turned number's products and sum by 2 u: 24 u of |a| + |b| in all, taken as 32 u. The angle is
off by 2^-52 of its fraction of a turn a position, the oracle's by 2^-53. Then one rounding to the
output's type, half of finfo.eps.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from oracle import q8, rope
from tests import q8_helpers as h

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _inputs(rng, B, T, Hq, H, D, dtype, packed=True):
    """Views q, k, v of one projection's output, and their values in fp64."""
    x = rng.normal(size=(B, T, Hq + 2 * H, D)) * np.exp(rng.normal(size=(Hq + 2 * H, D)) * 0.5)
    x = torch.from_numpy(x).to(TYPES[dtype]).cuda()
    parts = x.split([Hq, H, H], 2)
    if not packed:
        parts = [p.contiguous() for p in parts]
    return parts, [p.double().cpu().numpy() for p in parts]


def _weights(rng, D, dtype, norm):
    if not norm:
        return (None, None), (None, None)
    w = [torch.from_numpy(1 + 0.3 * rng.normal(size=D)).to(TYPES[dtype]).cuda() for _ in range(2)]
    return w, [x.double().cpu().numpy() for x in w]


def _freq(pairs, base=10000.0):
    return sv.rope_frequencies(pairs, base)[0] if pairs else None


def _host(f):
    return None if f is None else f.cpu().numpy()


def _bound(y, reach, pos, dtype):
    angle = np.abs(np.asarray(pos, np.float64))[..., None, None] * 2 * np.pi * 2.0 ** -52
    return (32 * U + angle) * reach + torch.finfo(TYPES[dtype]).eps / 2 * np.abs(y) * 1.01 + 1e-40


def _check(got, y, reach, pos, dtype):
    got = got.double().cpu().numpy()
    off = np.abs(got - y)
    assert (off <= _bound(y, reach, pos, dtype)).all(), float((off / (reach + 1e-30)).max())


@pytest.mark.parametrize("B,T,Hq,H,D,pairs,dtype,interleaved,norm", [
    (1, 1, 32, 8, 128, 64, "bf16", False, True),
    (3, 5, 32, 8, 128, 64, "bf16", True, True),
    (2, 37, 7, 1, 128, 32, "bf16", False, True),     # half of the head turned
    (2, 16, 12, 2, 64, 32, "fp32", True, False),
    (3, 17, 4, 4, 64, 32, "fp32", False, True),
    (2, 3, 5, 3, 256, 128, "bf16", False, True),
    (2, 3, 5, 3, 256, 128, "fp32", False, True),
    (1, 33, 28, 4, 80, 40, "bf16", False, True),
    (1, 33, 28, 4, 80, 20, "bf16", False, True),     # 8-byte vectors
    (1, 18, 28, 4, 80, 20, "fp32", True, True),
    (2, 5, 3, 2, 36, 18, "fp32", False, True),       # single numbers
    (2, 5, 3, 2, 102, 51, "bf16", False, True),
    (2, 5, 3, 2, 102, 33, "bf16", True, True),
    (2, 4, 3, 2, 2, 1, "fp32", False, True),
    (2, 4, 3, 2, 16, 0, "bf16", False, True),        # norm only
    (4, 9, 2, 1, 16, 8, "bf16", False, False),
    (300, 2, 2, 2, 32, 16, "bf16", False, True),
])
def test_heads(B, T, Hq, H, D, pairs, dtype, interleaved, norm):
    rng = np.random.default_rng(B * 1000 + T * 10 + D)
    (q, k, _), (qn, kn, _) = _inputs(rng, B, T, Hq, H, D, dtype)
    w, wn = _weights(rng, D, dtype, norm)
    f = _freq(pairs)
    L = rng.integers(0, 5000, B)
    pos = L[:, None] + np.arange(T)
    qo = torch.full((B, T, Hq, D), 7.0, dtype=TYPES[dtype], device="cuda")
    ko = torch.full((B, T, H, D), 7.0, dtype=TYPES[dtype], device="cuda")
    sv.qk_norm_rope(q, k, h.i32(L), qo, ko, inv_freq=f, rope_factor=1.25, interleaved=interleaved,
                    q_weight=w[0], k_weight=w[1], eps=1e-5)
    for got, x, g in ((qo, qn, wn[0]), (ko, kn, wn[1])):
        y, reach = rope.heads(x, g, pos, _host(f), interleaved=interleaved, factor=1.25, eps=1e-5)
        _check(got, y, reach, pos, dtype)


@pytest.mark.parametrize("far", [131071, (1 << 20) + 5, (1 << 30) - 3, -40])
def test_far_positions(far):
    rng = np.random.default_rng(5)
    (q, _, _), (qn, _, _) = _inputs(rng, 2, 3, 4, 1, 128, "fp32")
    f = _freq(64, 500000.0)
    pos = np.array([[far, 0, far - 1], [1, far, 2]])
    out = torch.empty((2, 3, 4, 128), device="cuda")
    sv.qk_norm_rope(q, None, None, out, None, inv_freq=f, positions=h.i32(pos))
    y, reach = rope.heads(qn, None, pos, _host(f))
    _check(out, y, reach, pos, "fp32")


def test_unusual_frequencies():
    """Many turns a position, negative, zero; what is not finite turns nothing."""
    f = torch.tensor([1000.0, -0.75, 0.0, 3e9, float("inf"), float("nan"), 1e-30, 6.2831855],
                     device="cuda")
    fn = np.where(np.isfinite(f.cpu().numpy()), f.cpu().numpy(), 0.0)
    rng = np.random.default_rng(6)
    (q, _, _), (qn, _, _) = _inputs(rng, 1, 5, 2, 1, 16, "fp32")
    out = torch.empty_like(q.contiguous())
    sv.qk_norm_rope(q, None, h.i32([0]), out, None, inv_freq=f)
    y, reach = rope.heads(qn, None, np.arange(5)[None], fn)
    # both angles are known to 2^-52 of themselves
    slack = 32 * U + np.abs(np.arange(5)[None, :, None, None] * np.tile(fn, 2)) * 2.0 ** -51
    assert (np.abs(out.double().cpu().numpy() - y) <= slack * reach + U * np.abs(y) + 1e-40).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 128), ("bf16", 36)])
def test_in_place_ragged_and_untouched(dtype, D):
    """q and k replaced within the projection's output; v, and tokens past num_new, stay."""
    rng = np.random.default_rng(8)
    B, T, Hq, H = 3, 6, 6, 2
    (q, k, v), (qn, kn, _) = _inputs(rng, B, T, Hq, H, D, dtype)
    v0, q0, k0 = v.clone(), q.clone(), k.clone()
    n = np.array([6, 0, 3])
    f = _freq(D // 2)
    L = np.array([0, 9, 77])
    pos = L[:, None] + np.arange(T)
    sv.qk_norm_rope(q, k, h.i32(L), q, k, inv_freq=f, num_new=h.i32(n))
    assert torch.equal(v, v0)
    for b in range(B):
        assert torch.equal(q[b, n[b]:], q0[b, n[b]:]) and torch.equal(k[b, n[b]:], k0[b, n[b]:])
        m = slice(0, n[b])
        for got, x in ((q, qn), (k, kn)):
            y, reach = rope.heads(x[b:b + 1, m], None, pos[b:b + 1, m], _host(f))
            _check(got[b:b + 1, m], y, reach, pos[b:b + 1, m], dtype)


def test_strides_that_vectors_do_not_fit():
    """An odd element offset and an odd token stride."""
    rng = np.random.default_rng(9)
    B, T, H, D = 2, 3, 2, 64
    buf = torch.from_numpy(rng.normal(size=1 + B * T * 131)).bfloat16().cuda()
    q = buf[1:].view(B * T, 131)[:, :H * D].view(B, T, H, D)
    out = torch.empty((B, T, H, D), dtype=torch.bfloat16, device="cuda")
    f = _freq(32)
    pos = np.array([[3, 4, 5], [10, 11, 12]])
    sv.qk_norm_rope(q, None, h.i32([3, 10]), out, None, inv_freq=f)
    y, reach = rope.heads(q.double().cpu().numpy(), None, pos, _host(f))
    _check(out, y, reach, pos, "bf16")


def test_bad_lengths_and_values():
    rng = np.random.default_rng(10)
    (q, k, _), (qn, _, _) = _inputs(rng, 4, 2, 2, 1, 32, "bf16", packed=False)
    q[3, 1, 0, 5] = float("nan")
    qo = torch.full_like(q, 3.0)
    ko = torch.full_like(k, 3.0)
    err = h.i32([0])
    sv.qk_norm_rope(q, k, h.i32([-1, 5, 5, 5]), qo, ko, inv_freq=_freq(16),
                    num_new=h.i32([2, 3, 2, 2]), q_weight=torch.ones(32, device="cuda").bfloat16(),
                    err_flag=err)
    assert int(err) == sv.SPEC_DERR_BAD_LENGTH
    assert (qo[:2] == 3).all() and (ko[:2] == 3).all() and not (ko[2:] == 3).all()
    assert torch.isnan(qo[3, 1, 0]).all() and torch.isfinite(qo[3, 1, 1]).all()
    assert torch.isfinite(qo[2]).all()


def test_binding_refuses_layouts():
    q = torch.zeros((2, 3, 4, 32), device="cuda")
    sl = h.i32([0, 0])
    ok = torch.zeros_like(q)
    f = _freq(16)
    for bad in (q.transpose(1, 2).contiguous().transpose(1, 2), q[:, :, :1].expand(2, 3, 4, 32),
                q[..., ::2].expand(2, 3, 4, 16), q[:, :2], q.bfloat16()):
        with pytest.raises((ValueError, TypeError)):
            sv.qk_norm_rope(q, None, sl, bad, None, inv_freq=f)
    for kw in (dict(inv_freq=f.double()), dict(inv_freq=f, q_weight=torch.ones(31, device="cuda")),
               dict(inv_freq=f, q_weight=torch.ones(32, device="cuda").bfloat16()),
               dict(inv_freq=f, positions=h.i32([[0, 0]])), dict(inv_freq=f, num_new=h.i32([1]))):
        with pytest.raises((ValueError, TypeError)):
            sv.qk_norm_rope(q, None, sl, ok, None, **kw)
    with pytest.raises(sv.SpecError):
        sv.qk_norm_rope(q, None, sl, ok, None, inv_freq=_freq(17))
    with pytest.raises(sv.SpecError):
        sv.qk_norm_rope(q, None, None, ok, None, inv_freq=f)


# ------------------------------------------------------------------ into the cache
def _append_case(seed, B, T, Hq, H, D, pairs, bs, dtype, *, interleaved=False, norm=True, lo=0,
                 hi=100, ragged=False, layers=2, tree=False, grow=1.0, scale_by=1.0):
    rng = np.random.default_rng(seed)
    (q, k, v), (qn, kn, vn) = _inputs(rng, B, T, Hq, H, D, dtype)
    w, wn = _weights(rng, D, dtype, norm)
    if grow != 1.0 and not norm:
        k.mul_(grow)
        kn = k.double().cpu().numpy()
    f = _freq(pairs)
    L = rng.integers(lo, hi + 1, B)
    n = rng.integers(0, T + 1, B) if ragged else np.full(B, T)
    bt, _, nb = h.table(rng, L + n, bs)
    pool, scales = h.cache(rng, nb, layers, H, bs, D)
    scales = scales * scale_by
    pos = L[:, None] + (rng.integers(0, T, (B, T)) if tree else np.arange(T))
    qo = torch.full((B, T, Hq, D), 5.0, dtype=TYPES[dtype], device="cuda")
    dp, ds, err = h.dev_pool(pool), h.dev_scales(scales), h.i32([0])
    sv.kv_q8_norm_rope_append(
        q, k, v, qo, dp, ds, h.i32(bt), h.i32(L), layer=layers - 1, inv_freq=f,
        interleaved=interleaved, q_weight=w[0], k_weight=w[1], rope_factor=1.1,
        positions=h.i32(pos) if tree else None, num_new=h.i32(n) if ragged else None, err_flag=err)
    assert int(err) == 0
    turn = dict(interleaved=interleaved, factor=float(np.float32(1.1)))
    y, reach = rope.heads(qn, wn[0], pos, _host(f), **turn)
    live = np.arange(T)[None, :] < n[:, None]
    ql = qo.double().cpu().numpy()
    assert (ql[~live] == 5).all()
    assert (np.abs(ql - y) <= _bound(y, reach, pos, dtype))[live].all()
    wp, wsc, _, ky, kreach = rope.append(kn, vn, pool, scales, bt, L, n, layer=layers - 1,
                                         weight=wn[1], positions=pos, inv_freq=_host(f), **turn)
    gp, gs = dp.view(torch.uint8).cpu().numpy(), ds.double().cpu().numpy()
    lay = layers - 1
    # other layers, values and their scales: the same bytes
    assert np.array_equal(gp[:, :lay], pool[:, :lay]) and np.array_equal(gs[:, :lay], scales[:, :lay])
    assert np.array_equal(gs[:, lay, 1], wsc[:, lay, 1])
    assert np.array_equal(gp[:, lay, 1], wp[:, lay, 1])
    # keys: a scale may differ only where the bound reaches over a power of two; a code is within
    # half a step (2^-4 of it, or 2^-10 scales) of the number that the oracle has
    touched = set()
    for b in range(B):
        at = int(L[b])
        while at < L[b] + n[b]:
            o = at % bs
            m = min(bs - o, int(L[b] + n[b]) - at)
            x = int(bt[b, at // bs])
            touched.add(x)
            rows = slice(at - int(L[b]), at - int(L[b]) + m)
            for hd in range(H):
                new, far = ky[b, rows, hd], kreach[b, rows, hd]
                slack = 33 * U * far
                s = gs[x, lay, 0, hd]
                was = scales[x, lay, 0, hd] if o else 0.0
                ok = {max(was, q8.block_scale(float((np.abs(new) + d * slack).max())))
                      for d in (-1, 1)}
                assert s in ok
                got = q8.VALUES[gp[x, lay, 0, hd, o:o + m]] * s
                assert (np.abs(got - new) <= np.maximum(np.abs(new) * 2.0 ** -4, s * 2.0 ** -10)
                        + 2 * slack).all()
                if s == wsc[x, lay, 0, hd]:
                    assert np.array_equal(gp[x, lay, 0, hd, :o], wp[x, lay, 0, hd, :o])
                    assert np.array_equal(gp[x, lay, 0, hd, o + m:], pool[x, lay, 0, hd, o + m:])
            at += m
    rest = [i for i in range(nb) if i not in touched]
    assert np.array_equal(gp[rest], pool[rest]) and np.array_equal(gs[rest], scales[rest])


@pytest.mark.parametrize("B,T,Hq,H,D,pairs,bs,dtype,more", [
    (1, 1, 32, 8, 128, 64, 16, "bf16", {}),
    (5, 5, 32, 8, 128, 64, 16, "bf16", {}),
    (3, 70, 4, 2, 128, 64, 16, "bf16", dict(ragged=True)),
    (3, 33, 8, 1, 64, 32, 16, "bf16", dict(interleaved=True)),
    (3, 15, 8, 2, 128, 32, 32, "bf16", dict(tree=True, norm=False)),
    (2, 90, 4, 2, 128, 64, 64, "bf16", dict(ragged=True)),        # more than a warp holds
    (2, 200, 2, 1, 64, 32, 128, "fp32", dict()),
    (2, 700, 1, 1, 32, 16, 512, "bf16", dict()),
    (1, 1500, 1, 1, 128, 64, 1024, "bf16", dict()),               # too long a table
    (2, 21, 7, 1, 80, 20, 8, "bf16", dict(interleaved=True)),
    (2, 21, 7, 1, 80, 13, 8, "fp32", dict()),                     # single numbers
    (2, 9, 3, 2, 256, 128, 16, "fp32", dict()),
    (2, 9, 3, 2, 256, 128, 16, "bf16", dict()),
    (2, 40, 3, 2, 16, 0, 16, "bf16", dict()),
    (3, 7, 3, 5, 48, 24, 5, "fp32", dict(ragged=True)),           # odd blocks
    (4, 5, 2, 2, 64, 32, 16, "bf16", dict(norm=False, grow=3000.0)),  # kept codes move
    (64, 5, 8, 2, 64, 32, 16, "bf16", dict(ragged=True)),
    # older scales between powers of two (a quotient of bf16 numbers by 1.5 2^e is a tie or at
    # least a third of a step from one: the values' codes are the oracle's)
    (5, 5, 4, 2, 128, 64, 64, "bf16", dict(lo=20, scale_by=1.5)),
    (3, 40, 4, 2, 64, 32, 128, "bf16", dict(lo=20, scale_by=96.0)),
])
def test_append(B, T, Hq, H, D, pairs, bs, dtype, more):
    _append_case(B * 31 + T, B, T, Hq, H, D, pairs, bs, dtype, **more)


def test_append_again_gives_the_same_bytes():
    rng = np.random.default_rng(3)
    (q, k, v), _ = _inputs(rng, 3, 20, 4, 2, 64, "bf16")
    L = np.array([5, 16, 40])
    bt, _, nb = h.table(rng, L + 20, 16)
    pool, scales = h.cache(rng, nb, 1, 2, 16, 64)
    dp, ds, qo = h.dev_pool(pool), h.dev_scales(scales), torch.empty_like(q.contiguous())
    args = (q, k, v, qo, dp, ds, h.i32(bt), h.i32(L))
    sv.kv_q8_norm_rope_append(*args, inv_freq=_freq(32))
    one = dp.view(torch.uint8).clone(), ds.clone(), qo.clone()
    sv.kv_q8_norm_rope_append(*args, inv_freq=_freq(32))
    assert torch.equal(dp.view(torch.uint8), one[0]) and torch.equal(ds, one[1])
    assert torch.equal(qo, one[2])


def test_append_errors_and_values():
    rng = np.random.default_rng(4)
    B, T, D = 4, 3, 64
    (q, k, v), (_, kn, vn) = _inputs(rng, B, T, 2, 2, D, "fp32", packed=False)
    k[3, 0, 0, 0] = float("inf")       # without a norm: its pair turns to infinities or NaN
    v[3, 1, 1, 3] = float("nan")
    v[3, 2, 0, 3] = -float("inf")
    L = np.array([-2, 31, 4, 10])
    bt = np.array([[0, 1], [2, 3], [99, 4], [5, 6]])
    pool, scales = h.cache(rng, 8, 1, 2, 16, D)
    dp, ds, err = h.dev_pool(pool), h.dev_scales(scales), h.i32([0])
    qo = torch.full_like(q, 9.0)
    sv.kv_q8_norm_rope_append(q, k, v, qo, dp, ds, h.i32(bt), h.i32(L), inv_freq=_freq(32),
                              err_flag=err)
    assert int(err) == sv.SPEC_DERR_BAD_LENGTH | sv.SPEC_DERR_BAD_BLOCK | sv.SPEC_DERR_VALUE
    assert (qo[:2] == 9).all() and not (qo[2:] == 9).any()
    gp, gs = dp.view(torch.uint8).cpu().numpy(), ds.cpu().numpy()
    assert np.array_equal(gp[:5], pool[:5]) and np.array_equal(gp[6:], pool[6:])
    vals = q8.VALUES[gp[5, 0]]
    assert np.isfinite(vals).all() and np.isfinite(gs).all()
    assert vals[1, 1, 11, 3] == 0 and vals[1, 0, 12, 3] * gs[5, 0, 1, 0] < -3e38 / 1.1


def test_values_that_are_not_finite_in_long_blocks():
    """Beyond what a warp holds at a time: zeros and the largest number, the others as ever."""
    rng = np.random.default_rng(13)
    T, D = 60, 128
    (q, k, v), (_, _, vn) = _inputs(rng, 1, T, 2, 1, D, "bf16", packed=False)
    v[0, 45, 0, 7], v[0, 3, 0, 9] = float("nan"), float("inf")
    k[0, 50, 0, 1] = float("nan")
    vn = v.double().cpu().numpy()
    pool, scales = h.cache(rng, 2, 1, 1, 64, D)
    dp, ds, err = h.dev_pool(pool), h.dev_scales(scales), h.i32([0])
    sv.kv_q8_norm_rope_append(q, k, v, torch.empty_like(q), dp, ds, h.i32([[1, 0]]), h.i32([0]),
                              k_weight=torch.ones(D, device="cuda").bfloat16(), err_flag=err)
    assert int(err) == sv.SPEC_DERR_VALUE
    wp, wsc, _ = q8.append(np.zeros((1, T, 1, D)), vn, pool, scales, np.array([[1, 0]]), [0])
    gp = dp.view(torch.uint8).cpu().numpy()
    assert np.array_equal(gp[1, 0, 1], wp[1, 0, 1]) and float(ds[1, 0, 1, 0]) == wsc[1, 0, 1, 0]
    keys = q8.VALUES[gp[1, 0, 0, 0]] * float(ds[1, 0, 0, 0])
    assert (keys[50] == 0).all() and np.isfinite(keys).all()
    y, _ = rope.heads(k.double().cpu().numpy(), np.ones(D), np.arange(T)[None], None)
    s = float(ds[1, 0, 0, 0])
    rows = [t for t in range(T) if t != 50]
    assert (np.abs(keys[rows] - y[0, rows, 0])
            <= np.maximum(np.abs(y[0, rows, 0]) * 2.0 ** -4, s * 2.0 ** -10) * 1.001).all()


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(12)
    (q, k, v), _ = _inputs(rng, 3, 5, 8, 2, 128, "bf16")
    L = np.array([5, 16, 40])
    bt, _, nb = h.table(rng, L + 5, 16)
    pool, scales = h.cache(rng, nb, 1, 2, 16, 128)
    f = _freq(64)
    tb, sl = h.i32(bt), h.i32(L)

    def run(out, dp, ds, stream=None):
        sv.kv_q8_norm_rope_append(q, k, v, out, dp, ds, tb, sl, inv_freq=f, stream=stream)

    want = torch.empty_like(q.contiguous()), h.dev_pool(pool), h.dev_scales(scales)
    run(*want)
    got = torch.empty_like(want[0]), h.dev_pool(pool), h.dev_scales(scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    run(*got, stream=side)
    side.synchronize()
    again = torch.empty_like(want[0]), h.dev_pool(pool), h.dev_scales(scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*again)
    graph.replay()
    torch.cuda.synchronize()
    for x in (got, again):
        for a, b in zip(x, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
