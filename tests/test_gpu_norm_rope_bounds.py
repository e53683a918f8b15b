"""Norms and rotary positions at the ends of their domain. The bound is that of
test_gpu_norm_rope.py."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from oracle import rope
from tests import q8_helpers as h
from tests.test_gpu_norm_rope import _check, _freq, _host, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(5, 128), (19, 36)])
def test_positions_past_32_bits(T, D):
    """The last length that there is: the tokens after it are at positions beyond the largest int."""
    rng = np.random.default_rng(1)
    (q, k, _), (qn, kn, _) = _inputs(rng, 2, T, 3, 2, D, "fp32")
    L = np.array([2 ** 31 - 3, 2 ** 31 - 1])
    pos = L[:, None] + np.arange(T)
    out = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    f = _freq(D // 2)
    sv.qk_norm_rope(q, k, h.i32(L), *out, inv_freq=f)
    for got, x in zip(out, (qn, kn)):
        y, reach = rope.heads(x, None, pos, _host(f))
        _check(got, y, reach, pos, "fp32")
