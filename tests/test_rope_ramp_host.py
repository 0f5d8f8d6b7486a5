"""Ramp scaling where the ramp lies outside the pairs: all pairs ahead of it turn as they are, all
behind it at 1 / factor."""

import math

import numpy as np
import pytest

import dequant_gemv_w4_amd as w4
import oracle


def _freqs(dim, base, original, low, high, factor=8.0):
    got, amplitude = w4.w4_rope_frequencies(w4.W4Rope.make(dim, base, scaling="ramp", factor=factor, low=low, high=high,
                                                           original_positions=original))
    assert math.isclose(amplitude, 1 + 0.1 * math.log(factor))
    ref, _ = oracle.rope_frequencies_ref(dim, base, "ramp", factor, low, high, original)
    assert np.allclose(got, ref, rtol=1e-13, atol=0)
    return np.array(got), base ** (-2 * np.arange(dim // 2) / dim)


@pytest.mark.parametrize("dim", [16, 64, 128])
def test_every_pair_turns_too_seldom(dim):
    # one position: even the first pair makes 1 / (2 pi) turns
    got, plain = _freqs(dim, 10000.0, 1, 1.0, 32.0)
    assert np.allclose(got, plain / 8, rtol=1e-13, atol=0)


@pytest.mark.parametrize("dim", [16, 64, 128])
def test_every_pair_turns_often(dim):
    # a small base: the last pair makes thousands of turns over the trained positions
    got, plain = _freqs(dim, 1.5, 1 << 20, 1.0, 32.0)
    assert (1 << 20) * plain[-1] / (2 * math.pi) > 1000
    assert np.allclose(got, plain, rtol=1e-13, atol=0)


def test_ramp_within_the_pairs_is_what_it_was():
    got, plain = _freqs(128, 10000.0, 4096, 1.0, 32.0, factor=16.0)
    a, b = (128 * math.log(4096 / (2 * math.pi * t)) / (2 * math.log(10000.0)) for t in (32.0, 1.0))
    r = np.clip((np.arange(64) - math.floor(a)) / (math.ceil(b) - math.floor(a)), 0, 1)
    assert 0 < r[25] < 1 and np.allclose(got, plain * (1 - r + r / 16), rtol=1e-13, atol=0)
