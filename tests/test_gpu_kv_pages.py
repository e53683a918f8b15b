"""kv_reserve, kv_fork and kv_free against the plain oracle (exact)."""
import numpy as np
import pytest

from gpu_helpers import gpu_lib
from oracle import pages
from q8_helpers import cache, dev_pool, dev_scales, i32, table

pytestmark = pytest.mark.gpu


def _stack(left, nb):
    fs = np.full(nb, -1, np.int64)
    fs[:len(left)] = left
    return fs, len(left)


def _state(rng, lengths, bs, mb, spare):
    bt, left, nb = table(rng, lengths, bs, mb, spare)
    fs, ft = _stack(left, nb)
    return dict(bt=bt, sl=np.array(lengths), refs=np.zeros(nb, np.int64), fs=fs, ft=ft, nb=nb)


def _same(got, want, names):
    for k in names:
        g = got[k].cpu().numpy()
        assert np.array_equal(g.reshape(np.shape(want[k])), want[k]), k


# ------------------------------------------------------------------ reserve
def _reserve(sv, s, n, bs, num_new=None):
    import torch
    d = {k: i32(s[k]) for k in ("bt", "sl", "fs")}
    ft, st = i32([s["ft"]]), i32([-9])
    sv.kv_reserve(d["bt"], d["sl"], d["fs"], ft, st, n=n, block_size=bs, num_blocks=s["nb"],
                  num_new=None if num_new is None else i32(num_new))
    torch.cuda.synchronize()
    want = pages.reserve(s["bt"], s["sl"], s["fs"], s["ft"], n, block_size=bs,
                         num_blocks=s["nb"], num_new=num_new)
    assert int(st.item()) == want["err"]
    _same(dict(block_table=d["bt"], free_top=ft), want, ("block_table", "free_top"))
    assert np.array_equal(d["fs"].cpu().numpy(), s["fs"])
    assert np.array_equal(d["sl"].cpu().numpy(), s["sl"])
    return want


@pytest.mark.parametrize("B,bs,n", [(1, 16, 1), (7, 1, 5), (256, 16, 5), (300, 4, 33),
                                    (1500, 16, 3), (8192, 8, 2), (5, 64, 2000)])
def test_reserve_matches_oracle(B, bs, n):
    rng = np.random.default_rng(B + bs)
    lengths = rng.integers(0, 5 * bs + 1, B)
    mb = -(-(5 * bs + n) // bs)
    s = _state(rng, lengths, bs, mb, B * (-(-n // bs) + 1))
    assert _reserve(gpu_lib(), s, n, bs)["err"] == 0
    nn = rng.integers(0, n + 1, B)
    # some rows hold blocks already
    for b in range(0, B, 3):
        j = -(-int(lengths[b]) // bs)
        if j < mb:
            s["ft"] -= 1
            s["bt"][b, j] = s["fs"][s["ft"]]
    assert _reserve(gpu_lib(), s, 0, bs, nn)["err"] == 0


def test_reserve_errors_change_nothing():
    sv = gpu_lib()
    rng = np.random.default_rng(2)
    base = _state(rng, [5, 16, 0, 31], 16, 4, 9)
    n = 20

    def change(**kw):
        s = {k: np.copy(v) if isinstance(v, np.ndarray) else v for k, v in base.items()}
        for k, v in kw.items():
            if isinstance(v, tuple):
                s[k][v[0]] = v[1]
            else:
                s[k] = v
        return s

    assert _reserve(sv, change(), n, 16)["err"] == 0
    assert _reserve(sv, change(sl=(1, -1)), n, 16)["err"] == pages.BAD_LENGTH
    assert _reserve(sv, change(sl=(1, 60)), n, 16)["err"] == pages.BAD_LENGTH
    assert _reserve(sv, change(), 0, 16, np.array([1, -1, 0, 0]))["err"] == pages.BAD_LENGTH
    assert _reserve(sv, change(ft=3), n, 16)["err"] == pages.NO_SPACE
    assert _reserve(sv, change(ft=-1), n, 16)["err"] == pages.NO_SPACE
    assert _reserve(sv, change(bt=((3, 2), base["nb"])), n, 16)["err"] == pages.BAD_BLOCK
    assert _reserve(sv, change(bt=((3, 2), -2)), n, 16)["err"] == pages.BAD_BLOCK
    assert _reserve(sv, change(fs=(base["ft"] - 1, -1)), n, 16)["err"] == pages.BAD_BLOCK


# ------------------------------------------------------------------ fork
def _fork(sv, s, src, dst, bs, *, layers=2, H=2, D=16, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    pool, scales = cache(rng, s["nb"], layers, H, bs, D)
    d = {k: i32(s[k]) for k in ("bt", "sl", "refs", "fs")}
    ft, st = i32([s["ft"]]), i32([-9])
    p, sc = dev_pool(pool), dev_scales(scales)
    sv.kv_fork(d["bt"], d["sl"], d["refs"], i32(src), i32(dst), p, d["fs"], ft, st, block_size=bs,
               kv_scales=sc)
    torch.cuda.synchronize()
    want = pages.fork(s["bt"], s["sl"], s["refs"], src, dst, s["fs"], s["ft"], block_size=bs,
                      num_blocks=s["nb"])
    assert int(st.item()) == want["err"]
    got = dict(block_table=d["bt"], seq_lens=d["sl"], extra_refs=d["refs"], free_top=ft)
    _same(got, want, got)
    for a, x, off in want["copies"] if want["err"] == 0 else ():
        pool[x, :, :, :, :off] = pool[a, :, :, :, :off]
        scales[x] = scales[a]
    assert np.array_equal(p.view(torch.uint8).cpu().numpy(), pool)
    assert np.array_equal(sc.double().cpu().numpy(), scales)
    # the other pool layout, same tables: [num_blocks, layers, 2, block_size, heads, dim] bf16
    d = {k: i32(s[k]) for k in ("bt", "sl", "refs", "fs")}
    ft = i32([s["ft"]])
    raw = rng.integers(-1000, 1000, (s["nb"], layers, 2, bs, H, D)).astype(np.int16)
    p = torch.from_numpy(raw.copy()).cuda().view(torch.bfloat16)
    sv.kv_fork(d["bt"], d["sl"], d["refs"], i32(src), i32(dst), p, d["fs"], ft, st, block_size=bs)
    torch.cuda.synchronize()
    assert int(st.item()) == want["err"]
    for a, x, off in want["copies"] if want["err"] == 0 else ():
        raw[x, :, :, :off] = raw[a, :, :, :off]
    assert np.array_equal(p.view(torch.int16).cpu().numpy(), raw)
    return want


@pytest.mark.parametrize("parents,children,bs", [(1, 1, 16), (1, 4, 16), (3, 40, 1), (8, 128, 16),
                                                 (20, 300, 4), (2, 9, 64)])
def test_fork_matches_oracle(parents, children, bs):
    rng = np.random.default_rng(parents * children)
    lengths = list(rng.integers(0, 6 * bs + 1, parents)) + [0] * children
    s = _state(rng, lengths, bs, 6, children + 3)
    s["refs"][s["bt"][0][s["bt"][0] >= 0]] = 2
    src = rng.integers(0, parents, children)
    dst = parents + rng.permutation(children)
    assert _fork(gpu_lib(), s, src, dst, bs)["err"] == 0


def test_fork_errors_change_nothing():
    sv = gpu_lib()
    rng = np.random.default_rng(3)
    base = _state(rng, [21, 40, 0, 0, 0], 16, 4, 4)

    def run(src, dst, **kw):
        s = {k: np.copy(v) if isinstance(v, np.ndarray) else v for k, v in base.items()}
        for k, v in kw.items():
            if isinstance(v, tuple):
                s[k][v[0]] = v[1]
            else:
                s[k] = v
        return _fork(sv, s, np.array(src), np.array(dst), 16, layers=1, H=1)["err"]

    assert run([0, 1], [2, 3]) == 0
    assert run([2], [3]) == 0                       # an empty parent
    assert run([0, 1], [2, 2]) == pages.BAD_SLOT    # a child twice
    assert run([0, 2], [2, 3]) == pages.BAD_SLOT    # a child that is a parent
    assert run([2], [2]) == pages.BAD_SLOT
    assert run([0, 5], [2, 3]) == pages.BAD_SLOT
    assert run([0, 0], [2, -1]) == pages.BAD_SLOT
    assert run([0], [1]) == pages.BAD_LENGTH        # a child that is in use
    assert run([0], [2], sl=(0, -3)) == pages.BAD_LENGTH
    assert run([0], [2], sl=(0, 65)) == pages.BAD_LENGTH
    assert run([0], [2], bt=((2, 1), 0)) == pages.BAD_BLOCK
    assert run([0], [2], bt=((0, 1), base["nb"])) == pages.BAD_BLOCK
    assert run([0, 1, 1], [2, 3, 4], ft=2) == pages.NO_SPACE
    assert run([0], [2], fs=(base["ft"] - 1, base["nb"])) == pages.BAD_BLOCK


# ------------------------------------------------------------------ free
def _shared(rng, parents, children, bs, mb, spare):
    """The state that forking leaves."""
    lengths = list(rng.integers(0, mb * bs + 1, parents)) + [0] * children
    s = _state(rng, lengths, bs, mb, children + spare)
    src = rng.integers(0, parents, children)
    w = pages.fork(s["bt"], s["sl"], s["refs"], src, parents + np.arange(children), s["fs"],
                   s["ft"], block_size=bs, num_blocks=s["nb"])
    assert w["err"] == 0
    s.update(bt=w["block_table"], sl=w["seq_lens"], refs=w["extra_refs"], ft=int(w["free_top"]))
    return s


def _free(sv, s, rows):
    import torch
    d = {k: i32(s[k]) for k in ("bt", "sl", "refs", "fs")}
    ft, st = i32([s["ft"]]), i32([-9])
    sv.kv_free(d["bt"], d["sl"], d["refs"], i32(rows), d["fs"], ft, st, num_blocks=s["nb"])
    torch.cuda.synchronize()
    want = pages.free(s["bt"], s["sl"], s["refs"], rows, s["fs"], s["ft"], num_blocks=s["nb"])
    assert int(st.item()) == want["err"]
    got = dict(block_table=d["bt"], seq_lens=d["sl"], extra_refs=d["refs"], free_stack=d["fs"],
               free_top=ft)
    _same(got, want, got)
    return want


@pytest.mark.parametrize("parents,children,bs,mb", [(1, 0, 16, 3), (1, 5, 16, 5), (4, 60, 1, 40),
                                                    (32, 224, 16, 256), (600, 1400, 4, 7)])
def test_free_matches_oracle(parents, children, bs, mb):
    rng = np.random.default_rng(parents + children)
    s = _shared(rng, parents, children, bs, mb, 3)
    n = parents + children
    assert _free(gpu_lib(), s, rng.permutation(n)[:max(1, n - 3)])["err"] == 0
    assert _free(gpu_lib(), s, rng.permutation(n))["err"] == 0
    assert _free(gpu_lib(), s, rng.permutation(n)[:1])["err"] == 0


def test_free_errors_change_nothing():
    sv = gpu_lib()
    rng = np.random.default_rng(4)
    base = _shared(rng, 3, 5, 4, 6, 2)
    base["sl"][0], base["bt"][0, 0] = max(base["sl"][0], 1), base["bt"][0, 0]

    def run(rows, **kw):
        s = {k: np.copy(v) if isinstance(v, np.ndarray) else v for k, v in base.items()}
        for k, v in kw.items():
            if isinstance(v, tuple):
                s[k][v[0]] = v[1]
            else:
                s[k] = v
        return _free(sv, s, np.array(rows))["err"]

    x = int(base["bt"][1][0])
    assert x >= 0
    assert run([1, 2]) == 0
    assert run([1, 1]) == pages.BAD_SLOT
    assert run([1, 8]) == pages.BAD_SLOT
    assert run([-1]) == pages.BAD_SLOT
    assert run([1], sl=(1, -5)) == pages.BAD_LENGTH
    assert run([1], bt=((1, 0), base["nb"])) == pages.BAD_BLOCK
    assert run([1], bt=((1, 0), -2)) == pages.BAD_BLOCK
    assert run([1], ft=-1) == pages.BAD_BLOCK
    # a block held once but listed by two rows
    assert run([1, 2], bt=((2, 5), x), refs=(x, 0)) in (0, pages.BAD_BLOCK)
    s = dict(base, bt=np.full((8, 6), -1), refs=np.zeros(base["nb"], int))
    s["bt"][1, 0] = s["bt"][2, 0] = x
    assert _free(sv, s, np.array([1, 2]))["err"] == pages.BAD_BLOCK
    # a stack without room: the ids on it are held twice
    assert run(list(range(8)), ft=base["nb"] - 1) == pages.BAD_BLOCK


# ------------------------------------------------------------------ long lists
# Lists above 8192 entries are planned by a cluster of CTAs, above 65536 in several rounds.
LONG = [(20, 900), (70, 2048)]


def _changed(s, **kw):
    s = {k: np.copy(v) if isinstance(v, np.ndarray) else v for k, v in s.items()}
    for k, (at, v) in kw.items():
        s[k][at] = v
    return s


@pytest.mark.parametrize("rows,blocks", LONG)
def test_reserve_long_lists(rows, blocks):
    sv = gpu_lib()
    rng = np.random.default_rng(rows)
    bs = 2
    lengths = rng.integers(0, 9, rows)
    s = _state(rng, lengths, bs, blocks, rows * blocks)
    for b in range(0, rows, 3):   # entries that hold a block already, here and there
        for j in rng.integers(6, blocks - 8, 20):
            if s["bt"][b, j] == -1:
                s["ft"] -= 1
                s["bt"][b, j] = s["fs"][s["ft"]]
    n = bs * (blocks - 6)
    assert _reserve(sv, s, n, bs)["err"] == 0
    assert _reserve(sv, s, 0, bs, rng.integers(0, n + 1, rows))["err"] == 0
    last = (rows - 1, blocks - 8)
    assert _reserve(sv, _changed(s, bt=(last, s["nb"])), n, bs)["err"] == pages.BAD_BLOCK
    assert _reserve(sv, _changed(s, sl=(rows - 1, -1)), n, bs)["err"] == pages.BAD_LENGTH
    assert _reserve(sv, dict(s, ft=rows * (blocks - 40)), n, bs)["err"] == pages.NO_SPACE
    assert _reserve(sv, _changed(s, fs=(s["ft"] - 9000, -1)), n, bs)["err"] == pages.BAD_BLOCK


@pytest.mark.parametrize("children,blocks", LONG)
def test_fork_long_lists(children, blocks):
    sv = gpu_lib()
    rng = np.random.default_rng(children)
    bs, parents = 2, 3
    lengths = [2 * blocks - 1, 2 * blocks, 2 * blocks - 301] + [0] * children
    s = _state(rng, lengths, bs, blocks, children + 3)
    src, dst = rng.integers(0, parents, children), parents + rng.permutation(children)
    small = dict(layers=1, H=1)
    assert _fork(sv, s, src, dst, bs, **small)["err"] == 0
    assert pages.BAD_SLOT == _fork(sv, s, src, np.append(dst[:-1], dst[0]), bs, **small)["err"]
    assert pages.BAD_SLOT == _fork(sv, s, np.append(src[:-1], dst[0]), dst, bs, **small)["err"]
    row, late = int(src[-1]), blocks - 200
    for kw in (dict(bt=((row, late), s["nb"])), dict(bt=((int(dst[-1]), late), 0))):
        assert _fork(sv, _changed(s, **kw), src, dst, bs, **small)["err"] == pages.BAD_BLOCK
    assert _fork(sv, dict(s, ft=3), src, dst, bs, **small)["err"] == pages.NO_SPACE
    assert _fork(sv, _changed(s, fs=(s["ft"] - 2, -1)), src, dst, bs, **small)["err"] == \
        pages.BAD_BLOCK


@pytest.mark.parametrize("children,blocks", LONG)
def test_free_long_lists(children, blocks):
    sv = gpu_lib()
    rng = np.random.default_rng(children)
    s = _shared(rng, 4, children, 2, blocks, 3)
    n = 4 + children
    rows = rng.permutation(n)
    assert _free(sv, s, rows)["err"] == 0
    assert _free(sv, s, rows[:n - 3])["err"] == 0
    # the undo of claims and counts
    assert _free(sv, s, np.append(rows[:-1], rows[0]))["err"] == pages.BAD_SLOT
    assert _free(sv, s, np.append(rows[:-1], n))["err"] == pages.BAD_SLOT
    held = int(s["bt"][rows[-1]][0])
    assert held >= 0
    assert _free(sv, _changed(s, refs=(held, 0)), rows)["err"] == pages.BAD_BLOCK
    assert _free(sv, _changed(s, bt=((rows[-1], blocks - 1), s["nb"])), rows)["err"] == \
        pages.BAD_BLOCK
    assert _free(sv, _changed(s, sl=(rows[-1], -2)), rows)["err"] == pages.BAD_LENGTH
    assert _free(sv, dict(s, ft=s["nb"] - 5), rows)["err"] == pages.BAD_BLOCK


def test_a_shared_prefix_lives_until_its_last_holder():
    """reserve, append, fork, attend and free together: children read their parent's tokens."""
    import torch
    sv = gpu_lib()
    rng = np.random.default_rng(5)
    B, MB, bs, NL, H, D, nb = 4, 8, 16, 1, 2, 128, 24
    bt, sl = i32(np.full((B, MB), -1)), i32(np.zeros(B))
    refs, fs, ft, st = i32(np.zeros(nb)), i32(rng.permutation(nb)), i32([nb]), i32([-1])
    pool = torch.zeros((nb, NL, 2, H, bs, D), dtype=torch.uint8, device="cuda").view(
        torch.float8_e4m3fn)
    scales = torch.zeros((nb, NL, 2, H), device="cuda")
    k, v = (torch.randn((B, 45, H, D), device="cuda").bfloat16() for _ in range(2))
    n = i32([45, 0, 0, 0])
    sv.kv_reserve(bt, sl, fs, ft, st, n=0, num_new=n, block_size=bs, num_blocks=nb)
    sv.kv_q8_append(k, v, pool, scales, bt, sl, num_new=n)
    sl += n
    sv.kv_fork(bt, sl, refs, i32([0, 0]), i32([2, 3]), pool, fs, ft, st, block_size=bs,
               kv_scales=scales)
    new = i32([1, 0, 1, 1])
    sv.kv_reserve(bt, sl, fs, ft, st, n=0, num_new=new, block_size=bs, num_blocks=nb)
    k1 = k[:, :1].contiguous()
    k1[1:] = k1[:1]
    sv.kv_q8_append(k1, k1, pool, scales, bt, sl, num_new=new)
    q = torch.randn((1, 1, 4, D), device="cuda").bfloat16().expand(B, 1, 4, D).contiguous()
    out = torch.empty_like(q)
    sv.kv_q8_attention(q, pool, scales, bt, sl, out, num_new=new)
    assert int(st.item()) == 0 and int(ft.item()) == nb - 3 - 2
    assert torch.equal(out[0], out[2]) and torch.equal(out[0], out[3])
    assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out.float()))
    for row, top in ((0, nb - 5 + 1), (3, nb - 5 + 2), (2, nb)):
        sv.kv_free(bt, sl, refs, i32([row]), fs, ft, st, num_blocks=nb)
        assert int(st.item()) == 0 and int(ft.item()) == top
    assert sorted(fs.cpu().tolist()) == list(range(nb)) and not torch.any(refs)
