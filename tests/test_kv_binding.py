"""What the binding of the cache operators keeps between calls and checks before a launch (CPU)."""
import pytest

import speculative_decoding_verification_sample_gb300 as sv


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verification_sample_gb300 import build
    build.build()
    sv._ready()


@pytest.fixture
def workspaces(monkeypatch):
    """The attention's kept workspaces, empty at first; a current stream 5 that captures or not."""
    import torch
    kept, state = {}, {"capturing": False}
    monkeypatch.setattr(sv, "_attn_workspaces", kept)
    monkeypatch.setattr(sv, "_raw_current", lambda index: 5)
    monkeypatch.setattr(sv, "_capturing", lambda: state["capturing"], raising=False)
    return kept, state, torch.device("cpu")


def test_first_call_sets_the_tested_name_last(monkeypatch):
    """Calls of other threads while one loads the library: what they test is set once everything
    that they use is."""
    names = ("_int32", "_float32", "_bfloat16", "_e4m3", "_uint8", "_raw_current", "_capturing",
             "_current_device", "_lib")
    for n in names:
        monkeypatch.setattr(sv, n, None, raising=False)
    load = sv.lib

    def slow():
        assert sv._int32 is None
        library = load()
        assert sv._int32 is None
        return library

    monkeypatch.setattr(sv, "lib", slow)
    assert sv._ready() is sv._lib
    assert all(getattr(sv, n) is not None for n in names)


SMALL, LARGE = (1, 4, 2, 64), (32, 4, 2, 128)


def test_workspace_is_kept_for_its_stream(workspaces):
    kept, _, dev = workspaces
    small = sv._attn_workspace(SMALL, dev, 5, None)
    assert sv._attn_workspace(SMALL, dev, 5, None)[:2] == small[:2]
    large = sv._attn_workspace(LARGE, dev, 5, None)
    # the larger one serves the smaller shape too
    assert sv._attn_workspace(SMALL, dev, 5, None)[2] is large[2]
    for (ptr, n, held), shape in ((small, SMALL), (large, LARGE)):
        assert ptr % 256 == 0 and n >= sv.kv_q8_attention_workspace_bytes(*shape)
        assert held.data_ptr() <= ptr and ptr + n <= held.data_ptr() + held.numel()
    assert sv._attn_workspace((33, 4, 2, 64), dev, 5, None)[:2] == (None, 0)


def test_workspace_of_a_capture_is_its_own(workspaces):
    """A graph holds its workspace's address for as long as it lives: what is kept for the calls
    to come, and is replaced by a larger one, must not be handed to it, nor its own be kept."""
    kept, state, dev = workspaces
    eager = sv._attn_workspace(SMALL, dev, 5, None)
    before = dict(kept)
    state["capturing"] = True
    one, two = (sv._attn_workspace(SMALL, dev, 5, None) for _ in range(2))
    large = sv._attn_workspace(LARGE, dev, 5, None)
    assert len({x[0] for x in (eager, one, two, large)}) == 4
    assert kept.keys() == before.keys() and all(kept[k] is before[k] for k in kept)
    state["capturing"] = False
    assert sv._attn_workspace(SMALL, dev, 5, None)[0] == eager[0]


# ------------------------------------------------------------------ checks of tensors
class OnDevice:
    """A CPU tensor that says it is on a CUDA device: what the binding looks at."""

    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda = t, index, True

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Library:
    """Notes the calls that would launch."""

    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    calls = []
    monkeypatch.setattr(sv, "_lib", Library(calls))
    monkeypatch.setattr(sv, "_raw_current", lambda index: 0)
    monkeypatch.setattr(sv, "_capturing", lambda: False, raising=False)
    monkeypatch.setattr(sv, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(sv, "_check", lambda t, name, ndim=None, dtype=None: _check(t, name, ndim,
                                                                                    dtype))
    return calls


def _check(t, name, ndim, dtype):
    if not getattr(t, "is_cuda", False) or not t.is_contiguous() or ndim not in (None, t.dim()):
        raise ValueError(name)
    if dtype not in (None, t.dtype):
        raise TypeError(name)


def _arguments():
    import torch
    i32, f32, bf16, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    z = lambda *s, dtype=i32: OnDevice(torch.zeros(s, dtype=dtype))  # noqa: E731
    pool, scales = z(4, 1, 2, 2, 16, 64, dtype=u8), z(4, 1, 2, 2, dtype=f32)
    table, lens = z(1, 2), z(1)
    blocks = dict(free_stack=z(4), free_top=z(1), status=z(1))
    return {
        "kv_q8_append": dict(k=z(1, 2, 2, 64, dtype=bf16), v=z(1, 2, 2, 64, dtype=bf16),
                             kv_pool=pool, kv_scales=scales, block_table=table, seq_lens=lens,
                             num_new=z(1), err_flag=z(1)),
        "kv_q8_attention": dict(q=z(1, 2, 4, 64, dtype=bf16), kv_pool=pool, kv_scales=scales,
                                block_table=table, seq_lens=lens, out=z(1, 2, 4, 64, dtype=bf16),
                                num_new=z(1), tree_mask=z(1, 2), workspace=z(1 << 10, dtype=u8),
                                err_flag=z(1)),
        "kv_reserve": dict(block_table=table, seq_lens=lens, num_new=z(1), **blocks),
        "kv_fork": dict(block_table=table, seq_lens=lens, extra_refs=z(4), src_rows=z(1),
                        dst_rows=z(1), kv_pool=pool, kv_scales=scales, **blocks),
        "kv_free": dict(block_table=table, seq_lens=lens, extra_refs=z(4), rows=z(1), **blocks),
    }


REST = {"kv_q8_append": {}, "kv_q8_attention": {}, "kv_reserve": dict(n=1, block_size=16, num_blocks=4),
        "kv_fork": dict(block_size=16), "kv_free": dict(num_blocks=4)}


@pytest.mark.parametrize("name", list(REST))
def test_every_tensor_must_be_on_the_current_device(calls, monkeypatch, name):
    f, ok = getattr(sv, name), _arguments()[name]
    f(**ok, **REST[name])
    assert calls == [name]
    for key, t in ok.items():
        for other in (OnDevice(t.t, 1), t.t):    # another device, the host
            with pytest.raises(ValueError):
                f(**{**ok, key: other}, **REST[name])
    monkeypatch.setattr(sv, "_current_device", lambda: 1)
    with pytest.raises(ValueError):
        f(**ok, **REST[name])
    assert calls == [name]


def test_stream_must_be_of_the_tensors_device(calls):
    class Stream:
        cuda_stream, device_index = 0, 1
    for name, ok in _arguments().items():
        with pytest.raises(ValueError):
            getattr(sv, name)(**ok, **REST[name], stream=Stream())
    assert calls == []


def test_workspace_is_checked_before_the_launch(calls):
    import torch
    ok = _arguments()["kv_q8_attention"]
    w = torch.zeros(1 << 10, dtype=torch.uint8)
    for err, bad in [(ValueError, w), (ValueError, OnDevice(w[::2])), (TypeError, OnDevice(w.int())),
                     (ValueError, OnDevice(w.view(32, 32))), (ValueError, OnDevice(w, 1))]:
        with pytest.raises(err):
            sv.kv_q8_attention(**{**ok, "workspace": bad})
    assert calls == []
