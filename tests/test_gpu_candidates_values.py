"""The example of shared prompts, its numbers: every step's cache and attention against the fp64
oracles, with the prompts' blocks shared (its prompts are too short for that to pay by itself)."""
import os

import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from oracle import q8, rope
from tests.gpu_helpers import ROOT, gpu_lib
from tests.test_gpu_norm_rope import _bound
from tests.test_gpu_prefix import check

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("kw", [dict(steps=4), dict(prompts=1, P=150, candidates=6, steps=3, K=1,
                                                    seed=3)])
def test_every_step(monkeypatch, kw):
    gpu_lib()
    monkeypatch.setenv("SPECVERIFY_SHARE", "1")
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    import q8_candidates
    append, attention = sv.kv_q8_norm_rope_append, sv.kv_q8_prefix_attention
    seen = dict(appends=0, shared=0, rows=0)

    def checked_append(q, k, v, q_out, pool, scales, table, lens, *, inv_freq, q_weight, k_weight,
                       num_new, err_flag):
        before = pool.view(torch.uint8).cpu().numpy(), _np(scales)
        append(q, k, v, q_out, pool, scales, table, lens, inv_freq=inv_freq, q_weight=q_weight,
               k_weight=k_weight, num_new=num_new, err_flag=err_flag)
        B, T = q.shape[:2]
        t, L = table.cpu().numpy(), lens.cpu().numpy()
        n = np.full(B, T) if num_new is None else num_new.cpu().numpy()
        live = np.arange(T)[None, :] < n[:, None]
        pos, f = L[:, None] + np.arange(T), inv_freq.cpu().numpy()
        y, reach = rope.heads(_np(q), _np(q_weight), pos, f)
        assert (np.abs(_np(q_out) - y) <= _bound(y, reach, pos, "bf16"))[live].all()
        want, wsc, _, ky, kreach = rope.append(_np(k), _np(v), *before, t, L, n, weight=_np(k_weight),
                                               positions=pos, inv_freq=f)
        codes, sc = pool.view(torch.uint8).cpu().numpy(), _np(scales)
        assert np.array_equal(codes[:, :, 1], want[:, :, 1])
        assert np.array_equal(sc[:, :, 1], wsc[:, :, 1])
        # a key is within half a step of the oracle's number (2^-4 of it, or 2^-10 scales), and
        # that off by what _bound says of fp32
        bs = pool.shape[4]
        for b, i in zip(*np.nonzero(live)):
            x, o = int(t[b, (L[b] + i) // bs]), int(L[b] + i) % bs
            for head in range(k.shape[2]):
                s = sc[x, 0, 0, head]
                off = np.abs(q8.VALUES[codes[x, 0, 0, head, o]] * s - ky[b, i, head])
                assert (off <= np.maximum(np.abs(ky[b, i, head]) * 2.0 ** -4, s * 2.0 ** -10)
                        + 2 * 33 * 2.0 ** -24 * kreach[b, i, head]).all()
        seen["appends"] += 1

    def checked_attention(q, pool, scales, table, lens, plan, out, *, num_new, err_flag):
        attention(q, pool, scales, table, lens, plan, out, num_new=num_new, err_flag=err_flag)
        n = None if num_new is None else num_new.cpu().numpy()
        check(out, _np(q), pool.view(torch.uint8).cpu().numpy(), _np(scales), table.cpu().numpy(),
              lens.cpu().numpy(), n)
        rows = torch.empty_like(out)
        sv.kv_q8_attention(q, pool, scales, table, lens, rows, num_new=num_new)
        seen["rows" if torch.equal(rows, out) else "shared"] += 1

    monkeypatch.setattr(sv, "kv_q8_norm_rope_append", checked_append)
    monkeypatch.setattr(sv, "kv_q8_prefix_attention", checked_attention)
    q8_candidates.main(**kw)
    pieces = -(-kw.get("P", 400) // 32)     # of the prompts, before there is anything to share
    assert seen == dict(appends=pieces + kw["steps"], rows=pieces, shared=kw["steps"])
