"""The oracle of norms and rotary positions against hand values and properties (CPU), and the
frequencies for long contexts."""
import math

import numpy as np
import pytest

from oracle import rope


def test_quarter_turn_by_hand():
    x = np.array([[[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]]])
    f = [math.pi / 2, math.pi]
    pos = np.array([[1]])
    y, _ = rope.heads(x, None, pos, f)
    assert np.allclose(y, [[[[-3, -2, 1, -4, 5, 6]]]])          # (1, 3) by 90, (2, 4) by 180 degrees
    y, _ = rope.heads(x, None, pos, f, interleaved=True, factor=2.0)
    assert np.allclose(y, [[[[-4, 2, -6, -8, 5, 6]]]])


def test_norm_by_hand():
    y, _ = rope.heads(np.array([[[[3.0, 4.0]]]]), [1.0, 2.0], np.array([[7]]), None, eps=0.0)
    assert np.allclose(y, [[[[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]]])


def test_products_depend_on_distances_only():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 1, 16))
    f = 100.0 ** (-np.arange(8) / 8)
    dot = lambda p, r: float((rope.heads(q, None, np.array([[p]]), f)[0]  # noqa: E731
                              * rope.heads(k, None, np.array([[r]]), f)[0]).sum())
    assert abs(dot(5, 2) - dot(905, 902)) < 1e-9


def test_frequencies():
    import speculative_decoding_verification_sample_gb300 as sv
    at = lambda *a, **k: sv.rope_frequencies(*a, device="cpu", **k)  # noqa: E731
    f, by = at(64, 10000.0)
    assert by == 1.0 and f[0] == 1.0 and abs(float(f[63]) - 10000.0 ** (-63 / 64)) < 1e-9
    assert np.allclose(at(64, scaling="linear", factor=4.0)[0], f / 4)
    b = at(64, scaling="base", factor=4.0)[0]
    assert b[0] == 1.0 and abs(float(b[63] / f[63]) - 0.25) < 1e-6
    p, by = at(64, scaling="parts", factor=4.0, trained_length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert abs(by - (0.1 * math.log(4) + 1)) < 1e-12
    assert np.allclose(p[turns >= 32], f[turns >= 32]) and np.allclose(p[turns <= 1],
                                                                      f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (p[mid] < f[mid]).all() and (p[mid] > f[mid] / 4).all()
    for bad in (dict(pairs=0), dict(pairs=4, base=0.0), dict(pairs=4, factor=-1.0),
                dict(pairs=4, scaling="other"),
                dict(pairs=4, scaling="parts", fast_turns=1.0, slow_turns=1.0)):
        with pytest.raises(ValueError):
            sv.rope_frequencies(device="cpu", **bad)
