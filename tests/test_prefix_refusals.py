"""Arguments that kv_prefix_plan and kv_q8_prefix_attention refuse before any launch (CPU)."""
import pytest

import speculative_decoding_verification_sample_gb300 as sv
from tests.test_kv_operators_refusals import EINVAL, ENOTSUP, P, L, _call  # noqa: F401

PLAN = dict(bt=P, sl=P, nn=None, starts=P, rows=P, NG=1, NE=2, T=3, Hq=4, H=2, NB=4, bs=16, B=2,
            MB=2, plan=P, pn=1 << 20, stream=None, err=None)
ATTN = dict(q=P, dtype=0, pool=P, scales=P, bt=P, sl=P, nn=None, tree=None, plan=P, pn=1 << 20,
            out=P, scale=0.125, NB=4, NL=2, layer=0, Hq=4, H=2, D=64, bs=16, B=1, T=3, MB=2, ws=P,
            wsn=1 << 30, stream=None, err=None)


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("bt", "sl", "starts", "rows", "plan")],
    *[(EINVAL, c) for c in (dict(NG=-1), dict(NE=-1), dict(T=0), dict(H=0), dict(Hq=3), dict(Hq=1),
                            dict(NB=0), dict(bs=0), dict(B=0), dict(MB=0), dict(MB=1 << 27),
                            dict(plan=P + 16), dict(pn=100))],
    *[(ENOTSUP, c) for c in (dict(B=8193), dict(NG=8193), dict(NE=8193), dict(T=33))],
])
def test_plan_refuses(L, want, changed):  # noqa: F811
    assert _call(L, "kv_prefix_plan", PLAN, **changed) == want


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("q", "out", "pool", "scales", "bt", "sl", "ws", "plan")],
    *[(EINVAL, c) for c in (dict(dtype=2), dict(scale=0.0), dict(scale=float("nan")),
                            dict(scale=float("inf")), dict(NB=0), dict(layer=2), dict(T=0),
                            dict(Hq=3), dict(B=0), dict(MB=0), dict(ws=P + 64), dict(wsn=100),
                            dict(plan=P + 8), dict(pn=200), dict(dtype=1, ws=None))],
    *[(ENOTSUP, c) for c in (dict(D=40), dict(T=33), dict(q=P + 8), dict(out=P + 8),
                             dict(pool=P + 8), dict(B=8193))],
])
def test_attention_refuses(L, want, changed):  # noqa: F811
    assert _call(L, "kv_q8_prefix_attention", ATTN, **changed) == want


def test_sizes(L):  # noqa: F811
    f = L.kv_prefix_plan_bytes
    assert f(4, 1, 4) > 0 and f(4, 1, 4) % 256 == 0 and f(400, 100, 300) > f(4, 1, 4)
    assert f(0, 1, 1) == f(1, -1, 1) == f(1, 1, -1) == f(8193, 1, 1) == 0
    assert f(1, 0, 0) > 0
    w = L.kv_q8_prefix_attention_workspace_bytes
    assert w(2, 5, 32, 8, 128) % 256 == 0
    assert w(1, 5, 32, 8, 96) >= L.kv_q8_attention_workspace_bytes(5, 32, 8, 96) > 0
    assert w(0, 5, 32, 8, 128) == w(2, 33, 32, 8, 128) == w(2, 5, 31, 8, 128) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    i = torch.zeros((1, 1), dtype=torch.int32)
    v = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.kv_prefix_plan(i, v, v, v, tokens=1, q_heads=2, kv_heads=1, block_size=16, num_blocks=1)
    with pytest.raises(ValueError):
        sv.kv_q8_prefix_attention(q, torch.zeros((2, 1, 2, 1, 16, 64), dtype=torch.uint8),
                                  torch.zeros((2, 1, 2, 1)), i, v, v, q)
