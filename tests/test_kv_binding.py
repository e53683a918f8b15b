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
