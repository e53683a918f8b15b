"""Attention of shared prefixes at the ends of its domain: waits that run out while products are in
flight, numbers near the ends of fp32, codes that are no numbers, the largest lists. The bounds are
those of test_gpu_prefix.py."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_sample_gb300 as sv
from tests import q8_helpers as h
from tests.test_gpu_prefix import _run, _small, check, plan_of, share  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T,groups", [(128, 4, ((5000, 40), (2000, 24))),   # two M tiles
                                        (64, 4, ((5000, 40), (2000, 24))),
                                        (128, 1, ((5000, 9), (2000, 5)))])    # one, in turns
def test_waits_run_out_with_products_in_flight(monkeypatch, D, T, groups):
    """The second group's keys are withheld where CTAs have the first group's products in flight:
    what is issued ends before the CTA does, and the next call is as ever."""
    _, L, bt, starts, members, nb, pool, scales, q, dq = _small(21, T=T, D=D, groups=groups)
    plan = plan_of(bt, L, starts, members, T, 8, 2, 16, nb)
    monkeypatch.setenv("SPECVERIFY_IDLE_NS", "5000000")
    for _ in range(3):
        err = h.i32([0])
        monkeypatch.setenv("SPECVERIFY_STALL_ROW", str(int(members[starts[1]])))
        _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == sv.SPEC_DERR_TIMEOUT
        monkeypatch.delenv("SPECVERIFY_STALL_ROW")
        err = h.i32([0])
        out = _run(dq, pool, scales, bt, L, plan, err_flag=err)
        assert int(err) == 0
        check(out, q, pool, scales, bt, L)
