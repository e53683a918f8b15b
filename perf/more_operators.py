"""Cases of the operators between a layer's projections and its attention over the 8-bit cache:
norms and rotary positions of queries and keys, the same with the keys and values written to the
8-bit paged cache, and attention of rows that share the blocks of a long prefix.

Rotation. Position p turns the pair i of a head's first 2 * len(inv_freq) numbers by the angle
p * inv_freq[i]: (a, b) -> f (a cos - b sin, b cos + a sin), f a common factor. The pair is
(i, i + len(inv_freq)) in the half layout, (2 i, 2 i + 1) in the interleaved one; the numbers after
the first 2 * len(inv_freq) stay. A norm, where there is a weight, comes first: x * weight /
sqrt(mean(x^2) + eps) over the whole head.

The cache is paged. Pool `[num_blocks, layers, 2, kv_heads, block_size, head_dim]` in e4m3 (plane 0
holds keys, plane 1 values) and one fp32 scale `[num_blocks, layers, 2, kv_heads]` for each block of
tokens and head: a cached number is code * scale. A row's logical position j lies in block
`block_table[b, j // block_size]` at offset `j % block_size`; unused table entries are -1.

With `own` false, `run` computes in elementary torch operations on fp32 (angles in fp64); with `own`
true it calls the package. The pool is returned as the e4m3 values it holds, next to their scales.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE_EXP = -100   # scales are powers of two in [2^-100, 2^120]
EPS = 1e-6
TILE = 1 << 22         # numbers of a piece of the plain forms' intermediate results


# ------------------------------------------------------------------ cases
def listed():
    w = dict(q_heads=32, kv_heads=8, head_dim=128)
    r = dict(op="rope", rot=128, interleaved=False, norm=True, dtype="bf16", scaling="none",
             tree=False)
    a = dict(op="append", rot=128, interleaved=False, norm=True, dtype="bf16", scaling="none",
             tree=False, ragged=False, block_size=16)
    p = dict(op="prefix", tree=False, layers=1, alone=0, block_size=16)
    return [
        # one sequence, one new token: latency
        dict(r, name="rope_one_token", rows=1, tokens=1, lo=400, hi=1000, **w),
        # the provisional tokens of the bench's batch, queries and keys of one layer
        dict(r, name="rope_verify_256", rows=256, tokens=5, lo=512, hi=4096, **w),
        # prompts of a few rows, interleaved pairs in the first half of the head, no norms
        dict(r, name="rope_prompts", rows=4, tokens=4099, lo=0, hi=700, **w,
             **{"rot": 64, "interleaved": True, "norm": False}),
        # fp32 activations, an odd group of heads, a rotated part that is not a power of two
        dict(r, name="rope_fp32_odd", rows=37, tokens=19, lo=0, hi=100000, q_heads=28, kv_heads=4,
             head_dim=80, **{"rot": 40, "dtype": "fp32", "scaling": "linear"}),
        # one sequence, one new token into the cache
        dict(a, name="append_one_token", rows=1, tokens=1, lo=400, hi=1000, **w),
        # the provisional tokens of the bench's batch into the cache of one layer
        dict(a, name="append_verify_256", rows=256, tokens=5, lo=512, hi=4096, **w),
        # prompts of a few rows, ragged lengths
        dict(a, name="append_prompts", rows=12, tokens=4099, lo=0, hi=700, **w,
             **{"ragged": True}),
        # draft trees far into a context scaled in parts, blocks of 32 tokens, no norms
        dict(a, name="append_tree", rows=48, tokens=15, lo=60000, hi=120000, q_heads=64,
             kv_heads=8, head_dim=128, **{"tree": True, "norm": False, "scaling": "parts",
                                          "block_size": 32}),
        # one prompt continued as four candidates, an early step: latency
        dict(p, name="prefix_four", groups=1, forks=4, plo=1000, phi=2000, lo=1, hi=64, tokens=5,
             **w),
        # eight prompts, sixteen candidates of each, two layers; two rows without company
        dict(p, name="prefix_candidates", groups=8, forks=16, plo=1024, phi=4096, lo=10, hi=300,
             tokens=5, **w, **{"layers": 2, "alone": 2}),
        # one long instruction before all the requests of a batch
        dict(p, name="prefix_instruction", groups=1, forks=256, plo=16000, phi=16384, lo=20,
             hi=600, tokens=5, **w),
        # draft trees of two prompts, wider groups of heads, blocks of 32 tokens
        dict(p, name="prefix_tree", groups=2, forks=24, plo=6000, phi=9000, lo=10, hi=500,
             tokens=16, q_heads=64, kv_heads=8, head_dim=128, **{"tree": True, "block_size": 32}),
    ]


def _span(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append", "append", "prefix", "prefix", "prefix"])
    kv, group = rng.choice([(8, 4), (8, 8), (4, 7), (16, 1), (2, 12), (1, 8)])
    c = dict(op=op, q_heads=kv * group, kv_heads=kv)
    if op == "prefix":
        tokens = _span(rng, 1, 32)
        groups = _span(rng, 1, 12)
        forks = _span(rng, 2, max(2, 256 // groups))
        # queries of a kv head times keys: no more than the largest listed case
        queries = groups * forks * tokens * group * kv
        phi = _span(rng, 40, max(80, min(32768, 256 * 5 * 32 * 16000 // (queries * groups))))
        c.update(groups=groups, forks=forks, tokens=tokens, plo=max(1, phi // 3), phi=phi, lo=0,
                 hi=_span(rng, 1, max(8, min(1000, 100000 // (groups * forks)))),
                 head_dim=rng.choice([64, 128, 128]), tree=rng.random() < 0.3,
                 layers=rng.choice([1, 1, 2]), alone=rng.choice([0, 0, 1, 3]),
                 block_size=rng.choice([16, 32, 64]))
        return c
    rows = _span(rng, 1, 256)
    heads = c["q_heads"] + 2 * kv
    tree = rng.random() < 0.25
    tokens = _span(rng, 1, 32 if tree else max(1, 12 * 4099 * 48 // (heads * rows)))
    if op == "rope":
        tokens = min(tokens, max(1, 4 * 4099 * 40 // (heads * rows)))
    dim = rng.choice([64, 80, 128, 128])
    c.update(rows=rows, tokens=tokens, lo=0, hi=_span(rng, 1, 1500 if op == "append" else 100000),
             head_dim=dim, rot=rng.choice([dim, dim, dim // 2, 16]),
             interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
             dtype=rng.choice(["bf16", "bf16", "fp32"]), tree=tree,
             scaling=rng.choice(["none", "none", "linear", "parts"]))
    if c["dtype"] == "fp32":
        c["tokens"] = max(1, tokens // 2)
    if op == "append":
        c.update(ragged=rng.random() < 0.5 and not tree, block_size=rng.choice([16, 32, 64]))
    return c


# ------------------------------------------------------------------ inputs
def _seeded(seed):
    g = torch.Generator(device="cuda").manual_seed(1000033 * seed + 29)
    return np.random.default_rng(6007 * seed + 11), g


def _int(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


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


def _frequencies(rot, scaling):
    """(inv_freq fp32, factor): radians a position of each pair, and the rotation's factor."""
    f = 500000.0 ** (-np.arange(0, rot, 2) / rot)
    factor = 1.0
    if scaling == "linear":            # positions eight times as dense
        f = f / 8
    elif scaling == "parts":           # fast pairs as they are, slow ones sixteen times denser
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1) / (32 - 1), 0, 1)
        f = f * keep + f / 16 * (1 - keep)
        factor = 0.1 * math.log(16) + 1
    return torch.from_numpy(f.astype(np.float32)).cuda(), factor


def _depths(rng, rows, tokens):
    """(parent of each token of a random draft tree, -1 for the first; depth)."""
    parent = np.full((rows, tokens), -1, np.int64)
    depth = np.zeros((rows, tokens), np.int64)
    for t in range(1, tokens):
        parent[:, t] = rng.integers(0, t, size=rows)
        depth[:, t] = depth[np.arange(rows), parent[:, t]] + 1
    return parent, depth


def _masks(parent):
    """Bit s of entry [b, t]: query t sees slot s, its own and its ancestors'."""
    rows, tokens = parent.shape
    m = np.ones((rows, tokens), np.int64)
    for t in range(1, tokens):
        m[:, t] = m[np.arange(rows), parent[:, t]] | (1 << t)
    return np.where(m >= 1 << 31, m - (1 << 32), m)


def _prepare_prefix(case, rng, g, s):
    """Groups of rows whose tables begin with the same blocks, as forking leaves them: the full
    blocks of the prefix are shared, the tail block and what follows are each row's own."""
    bs, T, D = case["block_size"], case["tokens"], case["head_dim"]
    G, F, B = case["groups"], case["forks"], case["groups"] * case["forks"] + case["alone"]
    pre = rng.integers(case["plo"], case["phi"] + 1, size=G)
    rows = rng.permutation(B)
    grouped = rows[:G * F].reshape(G, F)
    L = rng.integers(case["lo"], case["hi"] + 1, size=B)
    L[grouped] += pre[:, None]
    L[rows[G * F:]] += case["plo"]
    held = -(-(L + T) // bs)
    mb = int(held.max())
    shared = np.zeros(B, np.int64)
    shared[grouped] = (pre // bs)[:, None]
    nb = int((held - shared).sum() + (pre // bs).sum()) + 3
    ids, at = rng.permutation(nb), 0
    bt = np.full((B, mb), -1, np.int64)
    for i in range(G):
        n = int(pre[i] // bs)
        bt[grouped[i], :n] = ids[at:at + n]
        at += n
    for b in range(B):
        n = int(held[b] - shared[b])
        bt[b, shared[b]:held[b]] = ids[at:at + n]
        at += n
    s["pool"], s["scales"] = _cache(g, nb, case["layers"], case["kv_heads"], bs, D)
    s["q"] = torch.randn((case["layers"], B, T, case["q_heads"], D), device="cuda",
                         generator=g).bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["bt"], s["L"], s["nb"] = _int(bt), _int(L), nb
    s["starts"], s["members"] = _int(np.arange(G + 1) * F), _int(grouped.ravel())
    s["tree_mask"] = _int(_masks(_depths(rng, B, T)[0])) if case["tree"] else None


def prepare(case, seed):
    rng, g = _seeded(seed)
    s = dict(case)
    if case["op"] == "prefix":
        _prepare_prefix(case, rng, g, s)
        return s
    B, T, D = case["rows"], case["tokens"], case["head_dim"]
    Hq, H = case["q_heads"], case["kv_heads"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # the projection's output: queries, keys and values of a token side by side
    ch = torch.exp(torch.randn((Hq + 2 * H, D), device="cuda", generator=g) * 0.5)
    qkv = (torch.randn((B, T, Hq + 2 * H, D), device="cuda", generator=g) * ch).to(dt)
    s["q"], s["k"], s["v"] = qkv.split([Hq, H, H], 2)
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"], s["kw"] = (1 + 0.2 * torch.randn((2, D), device="cuda", generator=g)).to(dt)
    s["freq"], s["factor"] = _frequencies(case["rot"], case["scaling"])
    L = rng.integers(case["lo"], case["hi"] + 1, size=B)
    s["L"] = _int(L)
    s["pos"] = _int(L[:, None] + _depths(rng, B, T)[1]) if case["tree"] else None
    s["q_out"] = torch.empty((B, T, Hq, D), dtype=dt, device="cuda")
    if case["op"] == "rope":
        s["k_out"] = torch.empty((B, T, H, D), dtype=dt, device="cuda")
        return s
    bs = case["block_size"]
    n = rng.integers(T // 2, T + 1, size=B) if case["ragged"] else None
    # the table has the blocks that the new tokens touch; those before them are of no concern here
    first, held = L // bs, -(-(L + (T if n is None else n)) // bs)
    mb = max(1, int(held.max()))
    use = (np.arange(mb)[None, :] >= first[:, None]) & (np.arange(mb)[None, :] < held[:, None])
    nb = B * ((T + 2 * bs - 2) // bs) + 3   # what T tokens can touch at most
    bt = np.full((B, mb), -1, np.int64)
    bt[use] = rng.permutation(nb)[:int(use.sum())]
    s["pool"], s["scales"] = _cache(g, nb, 1, H, bs, D)
    s["bt"], s["n"] = _int(bt), (None if n is None else _int(n))
    if n is not None:
        s["q_out"].zero_()   # what lies behind a row's last token is left as it was
    return s


# ------------------------------------------------------------------ plain forms
def _positions(s):
    if s["pos"] is not None:
        return s["pos"].long()
    T = s["q"].shape[1]
    return s["L"].long()[:, None] + torch.arange(T, device=s["L"].device)[None, :]


def _turns(s):
    """cos and sin [B, T, 1, pairs], times the factor; the angles in fp64."""
    ang = _positions(s).double()[..., None] * s["freq"].double()
    return ((torch.cos(ang) * s["factor"]).float()[:, :, None],
            (torch.sin(ang) * s["factor"]).float()[:, :, None])


def _plain_heads(s, x, w, cos, sin):
    """Norm and rotation of x [B, T, heads, D], in fp32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    half = cos.shape[-1]
    part, rest = x[..., :2 * half], x[..., 2 * half:]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :half], part[..., half:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([part, rest], -1)


def _plain_rope(s):
    cos, sin = _turns(s)
    return {"q": _plain_heads(s, s["q"], s["qw"], cos, sin).to(s["q"].dtype),
            "k": _plain_heads(s, s["k"], s["kw"], cos, sin).to(s["k"].dtype)}


def _plain_scale(amax):
    """The smallest power of two s with amax <= 448 s, from amax = m 2^e, 0.5 <= m < 1."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, MIN_SCALE_EXP))
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=MIN_SCALE_EXP))


def _plain_append(s):
    pool, bs = s["pool"], s["block_size"]
    B, T, H, D = s["k"].shape
    dev = pool.device
    cos, sin = _turns(s)
    q = _plain_heads(s, s["q"], s["qw"], cos, sin).to(s["q"].dtype)
    k = _plain_heads(s, s["k"], s["kw"], cos, sin)
    L = s["L"].long()
    n = s["n"].long() if s["n"] is not None else torch.full_like(L, T)
    if s["n"] is not None:
        new = torch.arange(T, device=dev)[None, :] < n[:, None]
        q = torch.where(new[:, :, None, None], q, s["q_out"])
    # the blocks that a row's new tokens touch: index L // bs and on
    J = (T + 2 * bs - 2) // bs
    j = torch.div(L, bs, rounding_mode="floor")[:, None] + torch.arange(J, device=dev)[None, :]
    used = (j * bs < (L + n)[:, None]) & (n > 0)[:, None]
    b, w = torch.nonzero(used, as_tuple=True)
    jj = j[b, w]
    page = s["bt"].long()[b, jj]
    pos = jj[:, None] * bs + torch.arange(bs, device=dev)[None, :]               # [N, bs]
    t = pos - L[b][:, None]
    new, old = (t >= 0) & (t < n[b][:, None]), t < 0
    tc = t.clamp(0, T - 1)
    x = torch.stack([k[b[:, None], tc], s["v"][b[:, None], tc].float()], 1)      # [N, 2, bs, H, D]
    x = x.permute(0, 1, 3, 2, 4)                                                 # [N, 2, H, bs, D]
    nm, om = new[:, None, None, :, None], old[:, None, None, :, None]
    codes = pool[:, 0].view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
    had = s["scales"][:, 0][page]                                                # [N, 2, H]
    scale = _plain_scale(torch.where(nm, x.abs(), torch.zeros_like(x)).amax((3, 4)))
    scale = torch.where(old.any(1)[:, None, None], torch.maximum(scale, had), scale)
    kept = codes * (had / scale)[..., None, None]
    y = torch.where(nm, x / scale[..., None, None], torch.where(om, kept, codes))
    pool[:, 0].view(torch.uint8)[page] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    s["scales"][:, 0][page] = scale
    return {"q": q, "pool": pool, "scales": s["scales"]}


def _plain_prefix(s):
    """Every row by itself, over its whole length: what a prefix is shared for is not seen in the
    result. A few rows at a time, as the keys of all in fp32 are tens of GB."""
    bs, pool = s["block_size"], s["pool"]
    NL, B, T, Hq, D = s["q"].shape
    H = s["kv_heads"]
    bt, L = s["bt"].long(), s["L"].long()
    S = bt.shape[1] * bs
    out = torch.empty_like(s["q"])
    step = max(1, 64 * TILE // (H * S * D))
    t = torch.arange(T, device=bt.device)[None, :, None]
    j = torch.arange(S, device=bt.device)[None, None, :]
    for layer in range(NL):
        for r in range(0, B, step):
            pages, Lr = bt[r:r + step].clamp(min=0), L[r:r + step, None, None]
            n = pages.shape[0]
            sc = s["scales"][:, layer][pages]                                    # [n, MB, 2, H]
            kv = pool[:, layer].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
            kv = kv * sc[..., None, None]
            k, v = (kv[:, :, i].permute(0, 2, 1, 3, 4).reshape(n, H, S, D) for i in (0, 1))
            q = s["q"][layer, r:r + step].float().view(n, T, H, Hq // H, D)
            z = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, H, -1, D), k.transpose(2, 3))
            z = z / math.sqrt(D)
            seen = j <= Lr + t
            if s["tree_mask"] is not None:
                bit = (s["tree_mask"][r:r + step].long()[:, :, None] >> (j - Lr).clamp(0, 31)) & 1
                seen = (j < Lr) | ((j < Lr + T) & (bit == 1))
            seen = seen[:, None, :, None, :].expand(n, H, T, Hq // H, S).reshape(n, H, -1, S)
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            p = torch.exp(z - z.amax(-1, keepdim=True))
            v = torch.where((j < Lr + T).reshape(n, 1, S, 1), v, torch.zeros_like(v))
            o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
            o = o.view(n, H, T, Hq // H, D).permute(0, 2, 1, 3, 4)
            out[layer, r:r + step] = o.reshape(n, T, Hq, D).to(out.dtype)
    return {"out": out}


# ------------------------------------------------------------------ one pass
def _own(s):
    import speculative_decoding_verification_sample_gb300 as sv
    if s["op"] == "prefix":
        # the plan of a step serves all of its layers
        plan = sv.kv_prefix_plan(s["bt"], s["L"], s["starts"], s["members"], tokens=s["tokens"],
                                 q_heads=s["q_heads"], kv_heads=s["kv_heads"],
                                 block_size=s["block_size"], num_blocks=s["nb"])
        for layer in range(s["layers"]):
            sv.kv_q8_prefix_attention(s["q"][layer], s["pool"], s["scales"], s["bt"], s["L"], plan,
                                      s["out"][layer], layer=layer, tree_mask=s["tree_mask"])
        return {"out": s["out"]}
    how = dict(inv_freq=s["freq"], rope_factor=s["factor"], positions=s["pos"],
               interleaved=s["interleaved"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
    if s["op"] == "rope":
        sv.qk_norm_rope(s["q"], s["k"], s["L"], s["q_out"], s["k_out"], **how)
        return {"q": s["q_out"], "k": s["k_out"]}
    sv.kv_q8_norm_rope_append(s["q"], s["k"], s["v"], s["q_out"], s["pool"], s["scales"], s["bt"],
                              s["L"], layer=0, num_new=s["n"], **how)
    return {"q": s["q_out"], "pool": s["pool"], "scales": s["scales"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "prefix": _plain_prefix}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, D = case["tokens"], case["head_dim"]
    Hq, H = case["q_heads"], case["kv_heads"]
    if case["op"] == "prefix":
        rows = case["groups"] * case["forks"] + case["alone"]
        pre, mine = (case["plo"] + case["phi"]) / 2, (case["lo"] + case["hi"]) / 2 + T
        keys = case["groups"] * pre + case["alone"] * case["plo"] + rows * mine
        each = 2 * H * D + (2 * H * 4 + 4) / case["block_size"]
        seen = rows * (pre + mine)
        return {"bytes": case["layers"] * (keys * each + 2 * rows * T * Hq * D * 2),
                "flops": case["layers"] * 4 * T * Hq * D * seen}
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["rows"] * T * (0.75 if case.get("ragged") else 1.0)
    flops = n * (Hq + H) * (3 * case["rot"] + (4 * D if case["norm"] else 0))
    if case["op"] == "rope":
        return {"bytes": n * (Hq + H) * D * 2 * e + 4 * case["rows"], "flops": flops}
    each = 2 * Hq * D * e + 2 * H * D * (e + 1)
    return {"bytes": n * each + n / case["block_size"] * 2 * H * 4, "flops": flops}


# ------------------------------------------------------------------ from the definitions, 64 bits
def _exact_heads(case, s, x, w):
    """Norm and rotation in 64 bits: the pairs as complex numbers, turned by exp(i angle)."""
    x = x.double()
    if w is not None:
        x = x * w.double() / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    B, T = x.shape[:2]
    t = torch.arange(T, device="cuda", dtype=torch.float64)
    p = s["pos"].double() if s["pos"] is not None else s["L"].double()[:, None] + t
    turn = torch.polar(torch.full_like(p, _factor(s))[..., None].expand(-1, -1, len(s["freq"])),
                       p[..., None] * s["freq"].double())[:, :, None, :]
    h = case["rot"] // 2
    x = x.clone()
    re, im = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["interleaved"] else \
        (slice(0, h), slice(h, 2 * h))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return x


def _factor(s):
    return float(np.float32(s["factor"]))  # what a call receives


def _e4m3_grid():
    """Every non-negative finite value of e4m3 (bias 7, 3 bits; the code 127 is NaN)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return torch.from_numpy(np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))).cuda()


def _round_e4m3(x, grid):
    """To the nearest of the grid, ties to the even code."""
    a = x.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    return torch.copysign(grid[torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)], x)


def _exact_append(case, s):
    B, T, bs = case["rows"], case["tokens"], case["block_size"]
    bt, L = s["bt"].cpu().numpy(), s["L"].cpu().numpy()
    n = s["n"].cpu().numpy() if s["n"] is not None else np.full(B, T)
    if int(np.sum(n // bs + 2)) > 20000:
        return None
    q = _exact_heads(case, s, s["q"], s["qw"])
    src = [_exact_heads(case, s, s["k"], s["kw"]), s["v"].double()]
    if s["n"] is not None:
        for b in range(B):
            q[b, n[b]:] = s["q_out"][b, n[b]:].double()
    pool, scales = s["pool"].double(), s["scales"].double()
    grid = _e4m3_grid()
    for b in range(B):
        at, end = int(L[b]), int(L[b] + n[b])
        while at < end:
            page, o = int(bt[b, at // bs]), at % bs
            m = min(bs - o, end - at)
            for i in (0, 1):
                x = src[i][b, at - L[b]:at - L[b] + m].transpose(0, 1)           # [H, m, D]
                top = x.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(MIN_SCALE_EXP, 200)
                e = torch.where(torch.exp2(e) * E4M3_MAX < top, e + 1, e)
                e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= top, e - 1, e)
                sc = torch.exp2(e.clamp(min=MIN_SCALE_EXP))
                if o:
                    was = scales[page, 0, i]
                    sc = torch.maximum(sc, was)
                    pool[page, 0, i, :, :o] = _round_e4m3(
                        pool[page, 0, i, :, :o] * (was / sc)[:, None, None], grid)
                pool[page, 0, i, :, o:o + m] = _round_e4m3(x / sc[:, None, None], grid)
                scales[page, 0, i] = sc
            at += m
    return {"q": q, "pool": pool, "scales": scales}


def _exact_prefix(case, s):
    NL, B, T, Hq, D = s["q"].shape
    if work(case)["flops"] > 1.5e12:
        return None
    H, bs = case["kv_heads"], case["block_size"]
    bt, L = s["bt"].cpu().numpy(), s["L"].cpu().numpy()
    masks = s["tree_mask"].cpu().numpy() if s["tree_mask"] is not None else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(L[b]) + T
        ids = torch.from_numpy(bt[b, :-(-n // bs)].astype(np.int64)).cuda()
        see = np.zeros((T, n), bool)
        for t in range(T):
            see[t, :L[b] + (t + 1 if masks is None else 0)] = True
            if masks is not None:
                m = int(masks[b, t])
                see[t, L[b]:] = [(m >> i) & 1 for i in range(T)]
        hide = torch.from_numpy(~see).cuda()[None, :, None, :]
        for layer in range(NL):
            c = s["pool"].view(torch.uint8)[ids, layer].view(torch.float8_e4m3fn).double()
            c = c * s["scales"][ids, layer].double()[:, :, :, None, None]
            c = c.permute(1, 2, 0, 3, 4).reshape(2, H, -1, D)[:, :, :n]
            q = s["q"][layer, b].double().view(T, H, Hq // H, D)
            z = torch.einsum("thgd,hjd->htgj", q, c[0]) / D ** 0.5
            w = torch.softmax(z.masked_fill(hide, -math.inf), -1)
            out[layer, b] = torch.einsum("htgj,hjd->thgd", w, c[1]).reshape(T, Hq, D)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_heads(case, s, s["q"], s["qw"]),
                "k": _exact_heads(case, s, s["k"], s["kw"])}
    return (_exact_append if case["op"] == "append" else _exact_prefix)(case, s)
