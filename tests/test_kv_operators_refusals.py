"""Arguments that the 8-bit cache and block operators refuse before any launch (CPU: the
library checks its arguments on the host, and the binding its tensors)."""
import ctypes

import pytest

import speculative_decoding_verification_sample_gb300 as sv

P = 1 << 20   # an aligned address that no refused call touches
OK, EINVAL, ENOTSUP = 0, -1, -3


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verification_sample_gb300 import build
    build.build()
    return sv.lib()


def _call(L, name, spec, **changed):
    args = dict(spec)
    for k, v in changed.items():
        assert k in args, k
        args[k] = v
    return getattr(L, name)(*args.values())


APPEND = dict(k=P, v=P, dtype=0, pool=P, scales=P, bt=P, sl=P, nn=None, NB=4, NL=2, layer=0, H=2,
              D=64, bs=16, B=1, T=3, MB=2, stream=None, err=None)
ATTN = dict(q=P, dtype=0, pool=P, scales=P, bt=P, sl=P, nn=None, tree=None, out=P, scale=0.125,
            window=0, sinks=0, NB=4, NL=2, layer=0, Hq=4, H=2, D=64, bs=16, B=1, T=3, MB=2, ws=P,
            wsn=1 << 30, stream=None, err=None)
RESERVE = dict(bt=P, sl=P, nn=None, n=2, NB=4, bs=16, B=1, MB=2, fs=P, ft=P, st=P, stream=None)
FORK = dict(bt=P, sl=P, refs=P, src=P, dst=P, n=1, pool=P, planes=4, token=64, scales=None, NB=4,
            bs=16, B=2, MB=2, fs=P, ft=P, st=P, stream=None)
FREE = dict(bt=P, sl=P, refs=P, rows=P, n=1, NB=4, B=2, MB=2, fs=P, ft=P, st=P, stream=None)


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("k", "v", "pool", "scales", "bt", "sl")],
    *[(EINVAL, c) for c in (dict(dtype=7), dict(NB=0), dict(NL=0), dict(layer=2), dict(layer=-1),
                            dict(H=0), dict(D=0), dict(bs=0), dict(B=0), dict(T=0), dict(MB=0),
                            dict(MB=1 << 27), dict(T=1 << 30))],
    *[(ENOTSUP, c) for c in (dict(D=40), dict(k=P + 8), dict(v=P + 2), dict(pool=P + 4))],
])
def test_append_refuses(L, want, changed):
    assert _call(L, "kv_q8_append", APPEND, **changed) == want


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("q", "out", "pool", "scales", "bt", "sl", "ws")],
    *[(EINVAL, c) for c in (dict(dtype=2), dict(scale=0.0), dict(scale=-1.0),
                            dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
                            dict(sinks=-1), dict(sinks=2), dict(NB=0), dict(layer=5), dict(T=0),
                            dict(Hq=3), dict(Hq=1), dict(B=0), dict(MB=0), dict(ws=P + 64),
                            dict(wsn=100))],
    *[(ENOTSUP, c) for c in (dict(D=40), dict(D=272), dict(T=33), dict(q=P + 8), dict(out=P + 8),
                             dict(pool=P + 8), dict(tree=P, window=4))],
])
def test_attention_refuses(L, want, changed):
    assert _call(L, "kv_q8_attention", ATTN, **changed) == want


def test_attention_workspace_size(L):
    f = L.kv_q8_attention_workspace_bytes
    assert f(5, 32, 8, 128) > 0 and f(5, 32, 8, 128) % 256 == 0
    for bad in ((0, 32, 8, 128), (33, 32, 8, 128), (5, 33, 8, 128), (5, 4, 8, 128), (5, 32, 0, 128),
                (5, 32, 8, 24), (5, 32, 8, 0), (5, 32, 8, 512)):
        assert f(*bad) == 0


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("bt", "sl", "fs", "ft", "st")],
    *[(EINVAL, c) for c in (dict(n=-1), dict(NB=0), dict(bs=0), dict(B=0), dict(MB=0))],
    (ENOTSUP, dict(B=8193)),
])
def test_reserve_refuses(L, want, changed):
    assert _call(L, "kv_reserve", RESERVE, **changed) == want


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("bt", "sl", "refs", "src", "dst", "pool", "fs", "ft", "st")],
    *[(EINVAL, c) for c in (dict(n=0), dict(planes=0), dict(token=0), dict(NB=0), dict(B=0))],
    *[(ENOTSUP, c) for c in (dict(token=24), dict(pool=P + 8), dict(n=8193),
                             dict(token=1 << 24, bs=16))],
])
def test_fork_refuses(L, want, changed):
    assert _call(L, "kv_fork", FORK, **changed) == want


@pytest.mark.parametrize("want,changed", [
    *[(EINVAL, {k: None}) for k in ("bt", "sl", "refs", "rows", "fs", "ft", "st")],
    *[(EINVAL, c) for c in (dict(n=0), dict(NB=0), dict(B=0), dict(MB=0))],
    (ENOTSUP, dict(n=8193)),
])
def test_free_refuses(L, want, changed):
    assert _call(L, "kv_free", FREE, **changed) == want


def test_binding_refuses_cpu_tensors():
    import torch
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    pool = torch.zeros((2, 1, 2, 1, 16, 64), dtype=torch.uint8)
    sc = torch.zeros((2, 1, 2, 1))
    i = torch.zeros((1, 1), dtype=torch.int32)
    v = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.kv_q8_attention(q, pool, sc, i, v, q)
    with pytest.raises(ValueError):
        sv.kv_q8_append(q, q, pool, sc, i, v)
    with pytest.raises(ValueError):
        sv.kv_reserve(i, v, v, v, v, n=1, block_size=16, num_blocks=1)
    with pytest.raises(ValueError):
        sv.kv_fork(i, v, v, v, v, pool, v, v, v, block_size=16, kv_scales=sc)
    with pytest.raises(ValueError):
        sv.kv_free(i, v, v, v, v, v, v, num_blocks=1)


def test_status_names(L):
    assert ctypes.string_at(L.spec_status_string(ENOTSUP)) == b"unsupported configuration"
