"""Arguments that qk_norm_rope and kv_q8_norm_rope_append refuse before any launch (CPU)."""
import pytest

import speculative_decoding_verification_sample_gb300 as sv
from tests.test_kv_operators_refusals import EINVAL, ENOTSUP, P, L, _call  # noqa: F401

HEADS = dict(q=P, qs=512, k=P, ks=256, dtype=0, qo=P, qos=256, ko=P, kos=128, qw=P, kw=P, eps=1e-6,
             freq=P, pairs=32, inter=0, factor=1.0, sl=P, pos=None, nn=None, Hq=4, H=2, D=64, B=1,
             T=3, stream=None, err=None)
APPEND = dict(q=P, qs=512, k=P, ks=512, v=P, vs=512, dtype=0, qo=P, qos=256, qw=P, kw=P, eps=1e-6,
              freq=P, pairs=32, inter=0, factor=1.0, pool=P, scales=P, bt=P, sl=P, pos=None,
              nn=None, NB=4, NL=2, layer=0, Hq=4, H=2, D=64, bs=16, B=1, T=3, MB=2, stream=None,
              err=None)
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("q", "qo", "k", "ko", "freq", "sl")],
    *[(EINVAL, c) for c in (dict(dtype=2), dict(D=0), dict(D=63), dict(pairs=33), dict(pairs=-1),
                            dict(pairs=0), dict(Hq=0), dict(H=0), dict(H=-1), dict(B=0), dict(T=0),
                            dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(factor=NAN),
                            dict(factor=INF), dict(qs=255), dict(ks=127), dict(qos=255),
                            dict(kos=0), dict(qs=-256))],
    *[(ENOTSUP, c) for c in (dict(D=258, qs=4096, ks=4096, qos=4096, kos=4096), dict(q=P + 1),
                             dict(ko=P + 1), dict(kw=P + 1), dict(dtype=1, qw=P + 2),
                             dict(B=1 << 16, T=1 << 16), dict(qs=1 << 40))],
])
def test_norm_rope_refuses(L, want, changed):  # noqa: F811
    assert _call(L, "qk_norm_rope", HEADS, **changed) == want


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("q", "qo", "k", "v", "pool", "scales", "bt", "sl", "freq")],
    (EINVAL, dict(sl=None, pos=P)),
    *[(EINVAL, c) for c in (dict(dtype=2), dict(layer=2), dict(layer=-1), dict(NB=0), dict(bs=0),
                            dict(MB=0), dict(T=0), dict(T=1 << 30), dict(H=0), dict(Hq=0),
                            dict(pairs=40), dict(vs=64), dict(eps=-1.0), dict(factor=INF))],
    *[(ENOTSUP, c) for c in (dict(D=40, pairs=4), dict(pool=P + 8), dict(v=P + 1), dict(D=272))],
])
def test_norm_rope_append_refuses(L, want, changed):  # noqa: F811
    assert _call(L, "kv_q8_norm_rope_append", APPEND, **changed) == want


def test_binding_refuses_cpu_tensors():
    import torch
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    pool = torch.zeros((2, 1, 2, 2, 16, 64), dtype=torch.uint8)
    i = torch.zeros((1, 1), dtype=torch.int32)
    v = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.qk_norm_rope(q, q, v, q, q)
    with pytest.raises(ValueError):
        sv.kv_q8_norm_rope_append(q, q, q, q, pool, torch.zeros((2, 1, 2, 2)), i, v)
