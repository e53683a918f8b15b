"""Several candidates for each prompt, decoded with drafts on an 8-bit paged cache whose prompt
blocks they share; all bookkeeping on the device.

A toy target model (random weights: one attention layer with normed queries and keys, rotary
positions and a vocabulary projection). The prompts are written once and forked (kv_fork); the
candidates begin with the prompt's likeliest tokens. Every step:

    kv_reserve              blocks for the K + 1 provisional tokens of each row
    kv_q8_norm_rope_append  norms and positions of queries and keys, keys and values to the cache
    kv_prefix_plan          which rows begin with the same blocks (once for all layers)
    kv_q8_prefix_attention  each prompt's blocks read once for all of its candidates, where that
                            saves time: not for the few short rows here (SPECVERIFY_SHARE=1, a
                            test knob, shares them all the same)
    spec_verify_greedy      the drafts against the target's logits
    kv_commit_inplace       the accepted length; blocks past it go back to the free stack

    python examples/q8_candidates.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_sample_gb300 as sv  # noqa: E402
from q8_cache_loop import BS, D, HKV, HQ, V, Cache, Model  # noqa: E402


def attend(cache, model, tokens, freq, weights, groups, num_new=None):
    """Logits of `tokens` [rows, T] at the rows' next positions; the lengths are not changed."""
    T = tokens.shape[1]
    sv.kv_reserve(cache.table, cache.lens, cache.free, cache.top, cache.status, n=T,
                  num_new=num_new, block_size=BS, num_blocks=cache.num_blocks)
    q, k, v = model.qkv(tokens)
    turned, out = torch.empty_like(q), torch.empty_like(q)
    sv.kv_q8_norm_rope_append(q, k, v, turned, cache.pool, cache.scales, cache.table, cache.lens,
                              inv_freq=freq, q_weight=weights[0], k_weight=weights[1],
                              num_new=num_new, err_flag=cache.err)
    plan = sv.kv_prefix_plan(cache.table, cache.lens, *groups, tokens=T, q_heads=HQ, kv_heads=HKV,
                             block_size=BS, num_blocks=cache.num_blocks, num_new=num_new,
                             err_flag=cache.err)
    sv.kv_q8_prefix_attention(turned, cache.pool, cache.scales, cache.table, cache.lens, plan, out,
                              num_new=num_new, err_flag=cache.err)
    return model.logits(tokens, out)


def main(prompts=2, P=400, candidates=4, steps=12, K=3, seed=1):
    model = Model(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    freq = sv.rope_frequencies(D // 2, 10000.0)[0]
    weights = torch.ones((2, D), device="cuda", dtype=torch.bfloat16)
    tokens = torch.randint(0, V, (prompts, P), device="cuda")
    rows = prompts * candidates
    cache = Cache(rows, P // BS + 16, prompts * (P // BS + 1) + 16 * rows)
    none = torch.zeros(1, **i32), torch.zeros(0, **i32)

    # the prompts, in pieces of at most 32 tokens; the other rows are still empty
    head = torch.zeros((rows, P), dtype=torch.long, device="cuda")
    head[:prompts] = tokens
    at = 0
    while at < P:
        piece = min(32, P - at)
        new = torch.zeros(rows, **i32)
        new[:prompts] = piece
        logits = attend(cache, model, head[:, at:at + piece].contiguous(), freq, weights, none, new)
        cache.lens += new
        at += piece
    # candidate 0 of a prompt goes on in its row, the others in forks of it
    last = logits[:prompts, piece - 1].topk(candidates).indices.T.flatten()
    cache.fork(torch.arange(prompts, **i32).repeat(candidates - 1),
               torch.arange(prompts, rows, **i32))
    groups = (torch.arange(0, rows + 1, candidates, **i32),
              torch.arange(rows, **i32).view(candidates, prompts).T.flatten().contiguous())

    got = [[x] for x in last.tolist()]
    out, acc = torch.empty((rows, K + 1), **i32), torch.zeros(rows, **i32)
    for _ in range(steps):
        drafts = last[:, None].expand(rows, K)  # a guess: the last token again
        logits = attend(cache, model, torch.cat([last[:, None], drafts], 1), freq, weights, groups)
        sv.spec_verify_greedy(logits, drafts.int().contiguous(), out, acc)
        sv.kv_commit_inplace(cache.table, cache.lens, acc, cache.free, cache.top, cache.status,
                             K=K, block_size=BS, num_blocks=cache.num_blocks)
        o, a = out.tolist(), acc.tolist()
        for r in range(rows):
            got[r] += o[r][:a[r] + 1]
        last = torch.tensor([g[-1] for g in got], device="cuda")
    assert int(cache.status) == 0 and int(cache.err) == 0
    assert cache.lens.tolist() == [P + len(g) - 1 for g in got]
    cache.release(torch.arange(rows, **i32))
    assert int(cache.status) == 0 and int(cache.top) == cache.num_blocks
    print(f"{rows} candidates of {prompts} prompts of {P} tokens: "
          f"{sum(map(len, got))} tokens in {steps} steps")
    return got


if __name__ == "__main__":
    main()
