"""The example's loop: reserve, append, attend, verify, commit, fork and free together."""
import os
import sys

import pytest

from gpu_helpers import ROOT, gpu_lib

pytestmark = pytest.mark.gpu


def test_drafts_do_not_change_the_greedy_tokens():
    gpu_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import q8_cache_loop
    same, rows = q8_cache_loop.main()
    # a draft step's scales come from more tokens at once, so a block's 8-bit codes may differ
    # in the last bit and a near-tie may fall the other way; most rows must not
    assert same >= rows - 1
