"""Cases of the 8-bit paged-cache operators: appending, attention, page reservation, fork and free.

The cache is paged. Pool `[num_blocks, layers, 2, kv_heads, block_size, head_dim]` in e4m3 (plane 0
holds keys, plane 1 values) and one fp32 scale `[num_blocks, layers, 2, kv_heads]` for each block of
tokens and head: a cached number is code * scale. A row's logical position j lies in block
`block_table[b, j // block_size]` at offset `j % block_size`; unused table entries are -1.

With `own` false, `run` computes in elementary torch operations on fp32; with `own` true it calls the
package. The pool is returned as the e4m3 values it holds, next to their scales.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE_EXP = -100   # scales are powers of two in [2^-100, 2^120]


# ------------------------------------------------------------------ cases
def listed():
    w = dict(q_heads=32, kv_heads=8, head_dim=128, block_size=16)
    return [
        # one sequence, one new token, a short prompt behind it: latency
        dict(name="attend_one_token", op="attend", rows=1, tokens=1, lo=400, hi=1000, window=0,
             sinks=0, tree=False, **w),
        # the verification step of the bench's batch: 256 rows, 4 drafts and the last token
        dict(name="attend_verify_256", op="attend", rows=256, tokens=5, lo=512, hi=4096, window=0,
             sinks=0, tree=False, **w),
        # two very long contexts: few rows, the work split over the sequence
        dict(name="attend_long_context", op="attend", rows=2, tokens=5, lo=100000, hi=131072,
             window=0, sinks=0, tree=False, **w),
        # sliding window with sinks over long contexts, wider groups of heads
        dict(name="attend_window_sinks", op="attend", rows=48, tokens=7, lo=6000, hi=24000,
             window=4096, sinks=4, tree=False, q_heads=64, kv_heads=8, head_dim=128, block_size=32),
        # the provisional tokens of the bench's batch written to the cache of one layer
        dict(name="append_verify_256", op="append", rows=256, tokens=5, lo=512, hi=4096,
             ragged=False, dtype="bf16", kv_heads=8, head_dim=128, block_size=16),
        # prompts of a few rows written to the cache of one layer, ragged lengths
        dict(name="append_prompts", op="append", rows=12, tokens=4099, lo=0, hi=700, ragged=True,
             dtype="bf16", kv_heads=8, head_dim=128, block_size=16),
        # blocks for the provisional tokens of the bench's batch
        dict(name="reserve_verify_256", op="reserve", rows=256, tokens=5, lo=512, hi=4096,
             ragged=False, block_size=16),
        # blocks for whole prompts
        dict(name="reserve_prompts", op="reserve", rows=64, tokens=4096, lo=0, hi=900,
             ragged=True, block_size=16),
        # one sequence continued as four candidates
        dict(name="fork_four", op="fork", sources=1, forks=4, lo=500, hi=2000, layers=32,
             kv_heads=8, head_dim=128, block_size=16),
        # eight prompts, sixteen candidates of each
        dict(name="fork_many", op="fork", sources=8, forks=128, lo=512, hi=4096, layers=32,
             kv_heads=8, head_dim=128, block_size=16),
        # finished candidates: some of their blocks are still held by others
        dict(name="free_few", op="free", sources=1, forks=6, freed=5, lo=500, hi=2000,
             block_size=16),
        # a whole batch with shared prefixes ends at once
        dict(name="free_batch", op="free", sources=32, forks=224, freed=200, lo=512, hi=4096,
             block_size=16),
    ]


def _span(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "reserve", "fork", "free"])
    bs = rng.choice([16, 32, 64])
    if op == "attend":
        kv, group = rng.choice([(8, 4), (8, 8), (4, 7), (16, 1), (2, 12), (1, 8)])
        rows, tokens = _span(rng, 1, 256), _span(rng, 1, 32)
        most = max(4, min(131072, 256 * 2000 * 8 // (rows * kv)))
        if tokens * group > 32:
            most = max(4, most * 32 // (tokens * group))
        hi = _span(rng, 3, most)
        lo = _span(rng, 1, hi) if rng.random() < 0.8 else 0
        window = _span(rng, 1, hi) if rng.random() < 0.4 else 0
        return dict(op=op, rows=rows, tokens=tokens, lo=lo, hi=hi, window=window,
                    sinks=rng.choice([0, 1, 4, 37]) if window else 0,
                    tree=not window and rng.random() < 0.3, q_heads=kv * group, kv_heads=kv,
                    head_dim=rng.choice([64, 128, 128]), block_size=bs)
    if op == "append":
        rows = _span(rng, 1, 256)
        tokens = _span(rng, 1, max(1, 40000 // rows))
        return dict(op=op, rows=rows, tokens=tokens, lo=0, hi=_span(rng, 1, 2000),
                    ragged=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    kv_heads=rng.choice([1, 4, 8]), head_dim=rng.choice([64, 128, 128]),
                    block_size=bs)
    if op == "reserve":
        rows = _span(rng, 1, 1024)
        return dict(op=op, rows=rows, tokens=_span(rng, 1, max(1, min(4096, 200000 // rows))),
                    lo=0, hi=_span(rng, 1, 4096), ragged=rng.random() < 0.5, block_size=bs)
    sources = _span(rng, 1, 24)
    forks = _span(rng, 1, 100 if op == "fork" else 230)
    c = dict(op=op, sources=sources, forks=forks, lo=0, hi=_span(rng, 1, 4096), block_size=bs)
    if op == "fork":
        c.update(layers=rng.choice([1, 6, 16]), kv_heads=rng.choice([2, 8]),
                 head_dim=rng.choice([64, 128]))
        c["hi"] = min(c["hi"], 1500)
        c["sources"] = min(sources, 8)
    else:
        c["freed"] = rng.randint(1, sources + forks)
    return c


# ------------------------------------------------------------------ inputs
def _seeded(seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    return np.random.default_rng(7919 * seed + 5), g


def _int(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _table(rng, held, max_blocks, num_blocks):
    """Rows of `held[b]` distinct blocks each, in a shuffled order; the ids left over."""
    ids = rng.permutation(num_blocks)
    bt = np.full((len(held), max_blocks), -1, np.int64)
    mask = np.arange(max_blocks)[None, :] < np.asarray(held)[:, None]
    n = int(mask.sum())
    bt[mask] = ids[:n]
    return bt, ids[n:]


def _cache(g, num_blocks, layers, heads, bs, dim):
    """Codes as appending leaves them (standard deviation about 64 of the 448 that e4m3 reaches)
    and power-of-two scales that vary from block to block."""
    pool = torch.empty((num_blocks, layers, 2, heads, bs, dim), dtype=torch.float8_e4m3fn,
                       device="cuda")
    flat, step = pool.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, device="cuda", generator=g) * 64).clamp_(-448, 448).to(
            torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(-7, -4, (num_blocks, layers, 2, heads), device="cuda",
                                      generator=g).float())
    return pool, scales


def _free_stack(left, num_blocks):
    fs = np.full(num_blocks, -1, np.int64)
    fs[:len(left)] = left
    return fs


def _tables(**host):
    """int32 tables that a call changes, in one buffer, and the copy they are restored from."""
    host = {k: np.ascontiguousarray(v, np.int32) for k, v in host.items()}
    buf = _int(np.concatenate([v.ravel() for v in host.values()]))
    out, o = {}, 0
    for k, v in host.items():
        out[k] = buf[o:o + v.size].view(v.shape)
        o += v.size
    return out, buf, buf.clone()


def _lengths(rng, case, n):
    return rng.integers(case["lo"], case["hi"] + 1, size=n)


def _ragged(rng, case, rows):
    t = case["tokens"]
    return rng.integers(t // 2, t + 1, size=rows) if case["ragged"] else None


def _tree_masks(rng, rows, tokens):
    """Visible provisional slots of every query of a random draft tree: slot 0 is the last
    committed token, slot 1 + i node i; a query sees its own slot and its ancestors'."""
    m = np.zeros((rows, tokens), np.int64)
    m[:, 0] = 1
    for t in range(1, tokens):
        parent = rng.integers(0, t, size=rows)
        m[:, t] = m[np.arange(rows), parent] | (1 << t)
    return m


def _as_int32(m):
    return np.where(m >= 1 << 31, m - (1 << 32), m)


def prepare(case, seed):
    rng, g = _seeded(seed)
    s = dict(case)
    op, bs = case["op"], case["block_size"]
    if op == "attend":
        B, T, D = case["rows"], case["tokens"], case["head_dim"]
        L = _lengths(rng, case, B)
        held = -(-(L + T) // bs)
        mb = -(-(case["hi"] + T) // bs)
        nb = int(held.sum()) + 3
        bt, _ = _table(rng, held, mb, nb)
        s["pool"], s["scales"] = _cache(g, nb, 1, case["kv_heads"], bs, D)
        s["q"] = torch.randn((B, T, case["q_heads"], D), device="cuda", generator=g).bfloat16()
        s["bt"], s["L"] = _int(bt), _int(L)
        s["tree_mask"] = _int(_as_int32(_tree_masks(rng, B, T))) if case["tree"] else None
        s["out"] = torch.empty_like(s["q"])
    elif op == "append":
        B, T, H, D = case["rows"], case["tokens"], case["kv_heads"], case["head_dim"]
        L, n = _lengths(rng, case, B), _ragged(rng, case, B)
        held = -(-(L + (T if n is None else n)) // bs)
        mb = -(-(case["hi"] + T) // bs)
        nb = B * mb + 3
        bt, _ = _table(rng, held, mb, nb)
        s["pool"], s["scales"] = _cache(g, nb, 1, H, bs, D)
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a few channels are larger than the others, as keys have them
        ch = torch.exp(torch.randn((H, D), device="cuda", generator=g) * 0.7)
        s["k"] = (torch.randn((B, T, H, D), device="cuda", generator=g) * ch).to(dt)
        s["v"] = torch.randn((B, T, H, D), device="cuda", generator=g).to(dt)
        s["bt"], s["L"] = _int(bt), _int(L)
        s["n"] = None if n is None else _int(n)
    elif op == "reserve":
        B, T = case["rows"], case["tokens"]
        L, n = _lengths(rng, case, B), _ragged(rng, case, B)
        held = -(-L // bs)
        mb = -(-(case["hi"] + T) // bs)
        nb = B * mb + 64
        bt, left = _table(rng, held, mb, nb)
        s["t"], s["buf"], s["saved"] = _tables(bt=bt, fs=_free_stack(left, nb), ft=[len(left)])
        s["L"], s["n"], s["nb"] = _int(L), (None if n is None else _int(n)), nb
        s["status"] = _int([0])
    else:
        S, F = case["sources"], case["forks"]
        L = _lengths(rng, case, S)
        held = -(-L // bs)
        mb = max(1, -(-case["hi"] // bs))
        src = rng.integers(0, S, size=F)
        nb = S * mb + F + 16
        bt, left = _table(rng, held, mb, nb)
        bt = np.concatenate([bt, np.full((F, mb), -1, np.int64)])
        seq = np.concatenate([L, np.zeros(F, np.int64)])
        refs = np.zeros(nb, np.int64)
        dst = S + rng.permutation(F)
        if op == "fork":
            s["pool"], s["scales"] = _cache(g, nb, case["layers"], case["kv_heads"], bs,
                                            case["head_dim"])
            s["src"], s["dst"] = _int(src), _int(dst)
        else:
            # the state that forking leaves: full blocks shared, a tail block of one's own
            full = L // bs
            top = len(left)
            for a, b in zip(src, dst):
                bt[b, :full[a]] = bt[a, :full[a]]
                np.add.at(refs, bt[a, :full[a]], 1)
                if L[a] % bs:
                    top -= 1
                    bt[b, full[a]] = left[top]
                seq[b] = L[a]
            left = left[:top]
            s["rows"] = _int(rng.permutation(S + F)[:case["freed"]])
        s["t"], s["buf"], s["saved"] = _tables(bt=bt, L=seq, refs=refs,
                                               fs=_free_stack(left, nb), ft=[len(left)])
        s["nb"], s["status"] = nb, _int([0])
    return s


# ------------------------------------------------------------------ plain forms
def _cdiv(a, b):
    return torch.div(a + (b - 1), b, rounding_mode="floor")


def _plain_attend(s):
    q, pool, bs = s["q"], s["pool"], s["block_size"]
    B, T, Hq, D = q.shape
    H = s["kv_heads"]
    bt = s["bt"].long()
    S = bt.shape[1] * bs
    pages = bt.clamp(min=0)
    sc = s["scales"][:, 0][pages]                                            # [B, MB, 2, H]
    kv = pool[:, 0].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * sc[..., None, None]
    k, v = (kv[:, :, i].permute(0, 2, 1, 3, 4).reshape(B, H, S, D) for i in (0, 1))
    qf = q.float().view(B, T, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    z = torch.matmul(qf, k.transpose(2, 3)) / math.sqrt(D)
    L = s["L"].long()[:, None, None]
    t = torch.arange(T, device=q.device)[None, :, None]
    j = torch.arange(S, device=q.device)[None, None, :]
    seen = j <= L + t
    if s["window"]:
        seen = seen & ((j > L + t - s["window"]) | (j < s["sinks"]))
    if s["tree_mask"] is not None:
        bit = (s["tree_mask"].long()[:, :, None] >> (j - L).clamp(0, 31)) & 1
        seen = (j < L) | ((j < L + T) & (bit == 1))
    seen = seen[:, None, :, None, :].expand(B, H, T, Hq // H, S).reshape(B, H, -1, S)
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    v = torch.where((j < L + T).reshape(B, 1, S, 1), v, torch.zeros_like(v))
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(B, H, T, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    return {"out": o.to(q.dtype)}


def _plain_scale(amax):
    """The smallest power of two s with amax <= 448 s, from amax = m 2^e, 0.5 <= m < 1."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, MIN_SCALE_EXP))
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=MIN_SCALE_EXP))


def _plain_append(s):
    pool, bs = s["pool"], s["block_size"]
    B, T, H, D = s["k"].shape
    dev = pool.device
    L = s["L"].long()
    n = s["n"].long() if s["n"] is not None else torch.full_like(L, T)
    # the blocks that a row's new tokens touch: index L // bs and on
    J = (T + 2 * bs - 2) // bs
    j = torch.div(L, bs, rounding_mode="floor")[:, None] + torch.arange(J, device=dev)[None, :]
    used = (j * bs < (L + n)[:, None]) & (n > 0)[:, None]
    b, w = torch.nonzero(used, as_tuple=True)
    jj = j[b, w]
    page = s["bt"].long()[b, jj]
    pos = jj[:, None] * bs + torch.arange(bs, device=dev)[None, :]           # [N, bs]
    t = pos - L[b][:, None]
    new = (t >= 0) & (t < n[b][:, None])
    old = t < 0
    tc = t.clamp(0, T - 1)
    x = torch.stack([s["k"][b[:, None], tc], s["v"][b[:, None], tc]], 1).float()  # [N, 2, bs, H, D]
    x = x.permute(0, 1, 3, 2, 4)                                             # [N, 2, H, bs, D]
    nm = new[:, None, None, :, None]
    om = old[:, None, None, :, None]
    codes = pool[:, 0].view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
    had = s["scales"][:, 0][page]                                            # [N, 2, H]
    amax = torch.where(nm, x.abs(), torch.zeros_like(x)).amax((3, 4))
    scale = _plain_scale(amax)
    scale = torch.where(old.any(1)[:, None, None], torch.maximum(scale, had), scale)
    kept = codes * (had / scale)[..., None, None]
    y = torch.where(nm, x / scale[..., None, None], torch.where(om, kept, codes))
    pool[:, 0].view(torch.uint8)[page] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    s["scales"][:, 0][page] = scale
    return {"pool": pool, "scales": s["scales"]}


def _plain_reserve(s):
    bs = s["block_size"]
    bt, fs, ft = s["t"]["bt"].long(), s["t"]["fs"].long(), s["t"]["ft"].long()
    L = s["L"].long()
    n = s["n"].long() if s["n"] is not None else torch.full_like(L, s["tokens"])
    j = torch.arange(bt.shape[1], device=bt.device)[None, :]
    want = (j >= _cdiv(L, bs)[:, None]) & (j < _cdiv(L + n, bs)[:, None]) & (bt < 0)
    rank = torch.cumsum(want.reshape(-1).long(), 0).view_as(bt) - 1
    got = fs[(ft - 1 - rank).clamp(0, fs.numel() - 1)]
    return {"block_table": torch.where(want, got, bt).int(), "free_top": (ft - want.sum()).int(),
            "status": torch.zeros_like(s["status"])}


def _plain_fork(s):
    bs, t, pool = s["block_size"], s["t"], s["pool"]
    bt, L, refs, fs, ft = (t[k].long() for k in ("bt", "L", "refs", "fs", "ft"))
    src, dst = s["src"].long(), s["dst"].long()
    j = torch.arange(bt.shape[1], device=bt.device)[None, :]
    full = torch.div(L[src], bs, rounding_mode="floor")
    off = L[src] - full * bs
    shared = j < full[:, None]
    row = torch.where(shared, bt[src], torch.full_like(bt[src], -1))
    refs = refs + torch.zeros_like(refs).index_add_(
        0, row.clamp(min=0).reshape(-1), shared.reshape(-1).long())
    tail = off > 0
    rank = torch.cumsum(tail.long(), 0) - 1
    fresh = fs[(ft - 1 - rank).clamp(0, fs.numel() - 1)]
    row = torch.where((j == full[:, None]) & tail[:, None], fresh[:, None], row)
    i = torch.nonzero(tail).view(-1)
    a = bt[src[i], full[i]]
    raw = pool.view(torch.uint8)
    keep = torch.arange(bs, device=bt.device)[None, :] < off[i][:, None]
    raw[fresh[i]] = torch.where(keep[:, None, None, None, :, None], raw[a], raw[fresh[i]])
    s["scales"][fresh[i]] = s["scales"][a]
    bt = bt.index_copy(0, dst, row)
    L = L.index_copy(0, dst, L[src])
    return {"block_table": bt.int(), "seq_lens": L.int(), "extra_refs": refs.int(),
            "free_top": (ft - tail.sum()).int(), "pool": pool, "scales": s["scales"],
            "status": torch.zeros_like(s["status"])}


def _plain_free(s):
    t = s["t"]
    bt, L, refs, fs, ft = (t[k].long() for k in ("bt", "L", "refs", "fs", "ft"))
    rows = s["rows"].long()
    ids = bt[rows].reshape(-1)
    held = ids >= 0
    ids0 = ids.clamp(min=0)
    count = torch.zeros_like(refs).index_add_(0, ids0, held.long())
    order = torch.arange(ids.numel(), device=ids.device)
    first = torch.full_like(refs, ids.numel()).scatter_reduce(
        0, ids0, torch.where(held, order, torch.full_like(order, ids.numel())), "amin")
    ends = count > refs
    push = held & ends[ids0] & (first[ids0] == order)
    place = ft + torch.cumsum(push.long(), 0) - 1
    # entries that are not pushed go to a place of their own past the end
    fs = torch.cat([fs, fs[:1]])
    fs[torch.where(push, place, torch.full_like(place, fs.numel() - 1))] = ids
    refs = torch.where(ends, torch.zeros_like(refs), refs - count)
    bt = bt.index_copy(0, rows, torch.full_like(bt[rows], -1))
    L = L.index_copy(0, rows, torch.zeros_like(L[rows]))
    return {"block_table": bt.int(), "seq_lens": L.int(), "extra_refs": refs.int(),
            "free_stack": fs[:-1].int(), "free_top": (ft + push.sum()).int(),
            "status": torch.zeros_like(s["status"])}


# ------------------------------------------------------------------ one pass
def _own(s):
    import speculative_decoding_verification_sample_gb300 as sv
    op = s["op"]
    if op == "attend":
        sv.kv_q8_attention(s["q"], s["pool"], s["scales"], s["bt"], s["L"], s["out"], layer=0,
                           window=s["window"], sinks=s["sinks"], tree_mask=s["tree_mask"])
        return {"out": s["out"]}
    if op == "append":
        sv.kv_q8_append(s["k"], s["v"], s["pool"], s["scales"], s["bt"], s["L"], layer=0,
                        num_new=s["n"])
        return {"pool": s["pool"], "scales": s["scales"]}
    t = s["t"]
    s["buf"].copy_(s["saved"])  # the tables as they were before the call
    if op == "reserve":
        sv.kv_reserve(t["bt"], s["L"], t["fs"], t["ft"], s["status"], n=s["tokens"],
                      num_new=s["n"], block_size=s["block_size"], num_blocks=s["nb"])
        return {"block_table": t["bt"], "free_top": t["ft"], "status": s["status"]}
    if op == "fork":
        sv.kv_fork(t["bt"], t["L"], t["refs"], s["src"], s["dst"], s["pool"], t["fs"], t["ft"],
                   s["status"], kv_scales=s["scales"], block_size=s["block_size"])
        return {"block_table": t["bt"], "seq_lens": t["L"], "extra_refs": t["refs"],
                "free_top": t["ft"], "pool": s["pool"], "scales": s["scales"],
                "status": s["status"]}
    sv.kv_free(t["bt"], t["L"], t["refs"], s["rows"], t["fs"], t["ft"], s["status"],
               num_blocks=s["nb"])
    return {"block_table": t["bt"], "seq_lens": t["L"], "extra_refs": t["refs"],
            "free_stack": t["fs"], "free_top": t["ft"], "status": s["status"]}


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "append": _plain_append, "reserve": _plain_reserve,
            "fork": _plain_fork, "free": _plain_free}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, bs = case["op"], case["block_size"]
    mean = (case["lo"] + case["hi"]) / 2
    if op == "attend":
        B, T, H, D = case["rows"], case["tokens"], case["kv_heads"], case["head_dim"]
        keys = mean + T
        if case["window"]:
            keys = min(keys, case["window"] + case["sinks"] + T)
        cache = B * keys * 2 * H * D + B * keys / bs * (2 * H * 4 + 4)
        return {"bytes": cache + 2 * B * T * case["q_heads"] * D * 2,
                "flops": 4 * B * T * case["q_heads"] * keys * D}
    if op == "append":
        n = case["rows"] * case["tokens"] * (0.75 if case["ragged"] else 1.0)
        e = 2 if case["dtype"] == "bf16" else 4
        each = 2 * case["kv_heads"] * case["head_dim"]
        return {"bytes": n * each * (e + 1) + n / bs * 2 * case["kv_heads"] * 4,
                "flops": 2 * n * each}
    if op == "reserve":
        pops = case["rows"] * case["tokens"] * (0.75 if case["ragged"] else 1.0) / bs
        return {"bytes": 8 * case["rows"] + 12 * pops + 8, "flops": 0}
    if op == "fork":
        plane = 2 * case["layers"] * case["kv_heads"]
        tail = case["forks"] * plane * ((bs - 1) / 2 * case["head_dim"] + 4)
        return {"bytes": 2 * tail + case["forks"] * (8 * mean / bs + 16), "flops": 0}
    return {"bytes": case["freed"] * (mean / bs * 16 + 8), "flops": 0}


# ------------------------------------------------------------------ from the definitions, 64 bits
def _exact_attend(case, s):
    B, T, bs, D = case["rows"], case["tokens"], case["block_size"], case["head_dim"]
    H = case["kv_heads"]
    G = case["q_heads"] // H
    bt, L = s["bt"].cpu().numpy(), s["L"].cpu().numpy()
    masks = s["tree_mask"].cpu().numpy() if s["tree_mask"] is not None else None
    out = torch.zeros((B, T, H, G, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(L[b]) + T
        ids = torch.from_numpy(bt[b, :-(-n // bs)].astype(np.int64)).cuda()
        sc = s["scales"][ids, 0].double()                                    # [P, 2, H]
        c = s["pool"].view(torch.uint8)[ids, 0].view(torch.float8_e4m3fn).double()
        c = (c * sc[:, :, :, None, None]).permute(1, 2, 0, 3, 4).reshape(2, H, -1, D)[:, :, :n]
        pos = np.arange(n)
        see = np.zeros((T, n), bool)
        for t in range(T):
            if masks is not None:
                m = int(masks[b, t])
                see[t, :L[b]] = True
                for i in range(T):
                    see[t, L[b] + i] = (m >> i) & 1
            else:
                p = int(L[b]) + t
                see[t] = pos <= p
                if case["window"]:
                    see[t] &= (pos > p - case["window"]) | (pos < case["sinks"])
        see = torch.from_numpy(see).cuda()
        q = s["q"][b].double().view(T, H, G, D)
        z = torch.einsum("thgd,hjd->htgj", q, c[0]) / D ** 0.5
        z = z.masked_fill(~see[None, :, None, :], -math.inf)
        out[b] = torch.einsum("htgj,hjd->thgd", torch.softmax(z, -1), c[1])
    return {"out": out.view(B, T, H * G, D)}


def _e4m3_grid():
    """Every non-negative finite value of e4m3 (bias 7, 3 bits; the code 127 is NaN)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def _round_e4m3(x):
    """To the nearest of the grid, ties to the even code."""
    grid = _e4m3_grid()
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    return np.copysign(grid[np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)], x)


def _exact_append(case, s):
    B, T, bs = case["rows"], case["tokens"], case["block_size"]
    bt, L = s["bt"].cpu().numpy(), s["L"].cpu().numpy()
    n = s["n"].cpu().numpy() if s["n"] is not None else np.full(B, T)
    if int(n.sum()) * case["kv_heads"] * case["head_dim"] > 6_000_000:
        return None
    pool = s["pool"].float().cpu().numpy().astype(np.float64)
    scales = s["scales"].cpu().numpy().astype(np.float64)
    kv = [s["k"].float().cpu().numpy().astype(np.float64),
          s["v"].float().cpu().numpy().astype(np.float64)]
    for b in range(B):
        at, end = int(L[b]), int(L[b] + n[b])
        while at < end:
            page, o = int(bt[b, at // bs]), at % bs
            m = min(bs - o, end - at)
            for i in (0, 1):
                x = kv[i][b, at - L[b]:at - L[b] + m].transpose(1, 0, 2)     # [H, m, D]
                top = np.abs(x).max((1, 2))
                with np.errstate(divide="ignore"):
                    e = np.where(top > 0, np.ceil(np.log2(top / E4M3_MAX)), MIN_SCALE_EXP)
                e = np.where(np.exp2(e) * E4M3_MAX < top, e + 1, e)
                e = np.where(np.exp2(e - 1) * E4M3_MAX >= top, e - 1, e)
                sc = np.exp2(np.maximum(e, MIN_SCALE_EXP))
                if o:
                    was = scales[page, 0, i]
                    sc = np.maximum(sc, was)
                    pool[page, 0, i, :, :o] = _round_e4m3(
                        pool[page, 0, i, :, :o] * (was / sc)[:, None, None])
                pool[page, 0, i, :, o:o + m] = _round_e4m3(x / sc[:, None, None])
                scales[page, 0, i] = sc
            at += m
    return {"pool": pool, "scales": scales}


def _exact_fork(case, s):
    """The copied numbers; what is held in whole numbers has no 64-bit value to compare with."""
    bs = case["block_size"]
    if s["pool"].numel() > 400_000_000:
        return None
    t = {k: v.cpu().numpy() for k, v in s["t"].items()}
    pool, scales = s["pool"].double(), s["scales"].double()
    top = int(t["ft"][0])
    for a in s["src"].cpu().numpy():
        full, off = divmod(int(t["L"][a]), bs)
        if off:
            top -= 1
            x, y = int(t["fs"][top]), int(t["bt"][a, full])
            pool[x, :, :, :, :off] = pool[y, :, :, :, :off]
            scales[x] = scales[y]
    return {"block_table": None, "seq_lens": None, "extra_refs": None, "free_top": None,
            "pool": pool, "scales": scales, "status": None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "fork":
        return _exact_fork(case, s)
    return None
