"""The example of shared prompts runs: cache, positions, plan, attention, verification, commit."""
import os
import sys

import pytest

from gpu_helpers import ROOT, gpu_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [{}, dict(prompts=1, P=130, candidates=6, steps=5, K=1, seed=3)])
def test_candidates_of_shared_prompts(kw):
    gpu_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import q8_candidates
    got = q8_candidates.main(**kw)
    steps = kw.get("steps", 12)
    assert len(got) == kw.get("prompts", 2) * kw.get("candidates", 4)
    assert all(len(g) > steps and all(0 <= t < q8_candidates.V for t in g) for g in got)
