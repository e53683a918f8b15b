"""Sizes beyond an int's range that qk_norm_rope and kv_q8_norm_rope_append refuse (CPU)."""
import pytest

from tests.test_kv_operators_refusals import EINVAL, L, _call  # noqa: F401
from tests.test_norm_rope_refusals import APPEND, HEADS


@pytest.mark.parametrize("pairs", [1 << 30, (1 << 31) - 1, -(1 << 31)])
def test_pairs_whose_double_is_no_int(L, pairs):  # noqa: F811
    assert _call(L, "qk_norm_rope", HEADS, pairs=pairs) == EINVAL
    assert _call(L, "kv_q8_norm_rope_append", APPEND, pairs=pairs) == EINVAL
