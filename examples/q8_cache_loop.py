"""Speculative decoding on an 8-bit paged cache, all bookkeeping on the device.

A toy target model (random weights: one attention layer over the cache and a vocabulary
projection) decodes greedily with drafts of K tokens. Every step:

    kv_reserve         blocks for the K + 1 provisional tokens of each row
    kv_q8_append       their keys and values, 8 bits each, a scale for each block and head
    kv_q8_attention    their attention over the cached sequence
    spec_verify_greedy the drafts against the target's logits
    kv_commit_inplace  the accepted length; blocks past it go back to the free stack

After the prompts each row is forked (kv_fork), so that two candidates share its full blocks,
and at the end all rows are released (kv_free). The drafts are the target's own next tokens
with some replaced, so that acceptance varies; the output should not depend on them, which is
what the script looks at: it decodes once with drafts and once without (K = 0). Rows may differ
where two logits nearly tie: the scale of a block that keeps committed tokens may have grown with
a rejected draft, which rounds the block's codes once more.

    python examples/q8_cache_loop.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_sample_gb300 as sv  # noqa: E402

V, HQ, HKV, D, BS = 4096, 8, 2, 128, 16


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        self.embed = r(V, HQ * D)
        self.wq = r(HQ * D, HQ * D) / (HQ * D) ** 0.5
        self.wk = r(HQ * D, HKV * D) / (HQ * D) ** 0.5
        self.wv = r(HQ * D, HKV * D) / (HQ * D) ** 0.5
        self.out = r(HQ * D, V) / (HQ * D) ** 0.5

    def qkv(self, tokens):
        x = self.embed[tokens]
        split = lambda w, h: (x @ w).view(*tokens.shape, h, D).bfloat16()  # noqa: E731
        return split(self.wq, HQ), split(self.wk, HKV), split(self.wv, HKV)

    def logits(self, tokens, attended):
        x = self.embed[tokens] + 4 * attended.float().flatten(-2)
        return x @ self.out


class Cache:
    def __init__(self, rows, max_blocks, num_blocks):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.pool = torch.zeros((num_blocks, 1, 2, HKV, BS, D), dtype=torch.uint8,
                                device="cuda").view(torch.float8_e4m3fn)
        self.scales = torch.zeros((num_blocks, 1, 2, HKV), device="cuda")
        self.table = torch.full((rows, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(num_blocks, dtype=torch.int32, device="cuda")
        self.free = torch.arange(num_blocks, dtype=torch.int32, device="cuda")
        self.top, self.status, self.err = i([num_blocks]), i([0]), i([0])
        self.num_blocks = num_blocks

    def step(self, model, tokens, num_new=None):
        """Logits of `tokens` [rows, T] at the rows' next positions; the length is not changed."""
        T = tokens.shape[1]
        sv.kv_reserve(self.table, self.lens, self.free, self.top, self.status, n=T,
                      num_new=num_new, block_size=BS, num_blocks=self.num_blocks)
        q, k, v = model.qkv(tokens)
        sv.kv_q8_append(k, v, self.pool, self.scales, self.table, self.lens, num_new=num_new,
                        err_flag=self.err)
        out = torch.empty_like(q)
        sv.kv_q8_attention(q, self.pool, self.scales, self.table, self.lens, out,
                           num_new=num_new, err_flag=self.err)
        return model.logits(tokens, out)

    def fork(self, src, dst):
        sv.kv_fork(self.table, self.lens, self.refs, src, dst, self.pool, self.free, self.top,
                   self.status, block_size=BS, kv_scales=self.scales)

    def release(self, rows):
        sv.kv_free(self.table, self.lens, self.refs, rows, self.free, self.top, self.status,
                   num_blocks=self.num_blocks)


def decode(model, prompts, steps, K, guess):
    """Greedy tokens [2 n, steps] of n prompts, each forked once. guess(row-wise last tokens, i)
    proposes K drafts; every step commits the accepted ones and the target's next token."""
    n, P = prompts.shape
    rows = 2 * n
    cache = Cache(rows, 64, 64 * rows)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = torch.cat([torch.full((n,), P - 1, **i32), torch.zeros(n, **i32)])
    head = torch.zeros((rows, P - 1), dtype=torch.long, device="cuda")
    head[:n] = prompts[:, :-1]
    at = 0
    while at < P - 1:  # the prompt but its last token, in pieces of at most 32 tokens
        piece = min(32, P - 1 - at)
        new = torch.cat([torch.full((n,), piece, **i32), torch.zeros(n, **i32)])
        cache.step(model, head[:, at:at + piece].contiguous(), num_new=new)
        cache.lens += new
        at += piece
    assert torch.equal(cache.lens, lens)
    cache.fork(torch.arange(n, **i32), torch.arange(n, rows, **i32))
    last = prompts[:, -1].repeat(2)
    got = [[] for _ in range(rows)]
    out = torch.empty((rows, K + 1), **i32)
    acc = torch.zeros(rows, **i32)
    while min(map(len, got)) < steps:
        drafts = guess([len(g) for g in got])
        tokens = torch.cat([last[:, None], drafts], 1) if K else last[:, None]
        logits = cache.step(model, tokens.long().contiguous())
        if K:
            sv.spec_verify_greedy(logits, drafts.int().contiguous(), out, acc)
        else:
            out[:, 0] = logits[:, 0].argmax(-1)
        sv.kv_commit_inplace(cache.table, cache.lens, acc, cache.free, cache.top, cache.status,
                             K=K, block_size=BS, num_blocks=cache.num_blocks)
        o, a = out.tolist(), acc.tolist()
        for r in range(rows):
            got[r] += o[r][:a[r] + 1]
        last = torch.tensor([g[-1] for g in got], device="cuda")
    assert int(cache.status) == 0 and int(cache.err) == 0
    cache.release(torch.randperm(rows, device="cuda").int())
    assert int(cache.status) == 0 and int(cache.top) == cache.num_blocks
    assert sorted(cache.free.tolist()) == list(range(cache.num_blocks)) and not cache.refs.any()
    return [g[:steps] for g in got]


def main(n=3, P=70, steps=40, K=4, seed=1):
    model = Model(seed)
    prompts = torch.randint(0, V, (n, P), device="cuda")
    plain = decode(model, prompts, steps + K + 1, 0, lambda at: None)
    assert plain[:n] == plain[n:]  # a fork continues as its parent does
    wrong = torch.Generator().manual_seed(seed)

    def guess(at):
        d = [[plain[r][min(i + x, len(plain[r]) - 1)] for x in range(K)] for r, i in enumerate(at)]
        d = torch.tensor(d)
        miss = torch.rand(d.shape, generator=wrong) < 0.3
        return torch.where(miss, (d + 1) % V, d).cuda()

    drafted = decode(model, prompts, steps, K, guess)
    same = sum(a == b[:steps] for a, b in zip(drafted, plain))
    print(f"{same} of {2 * n} rows decode the same tokens with drafts as without")
    return same, 2 * n


if __name__ == "__main__":
    main()
