"""Rotary plans at their ends: what Rope.build says of the pairs of a yarn plan holds for every pair, whatever
the original length.  No GPU."""
import math

import numpy as np
import pytest

from test_sequence_modeling_b200 import ttt


@pytest.mark.parametrize("length", [1, 4, 6, 7, 60, 200, 300, 4096, 10 ** 7, 10 ** 12])
@pytest.mark.parametrize("rotary", [2, 4, 16, 64])
@pytest.mark.parametrize("betas", [(32.0, 1.0), (1.5, 1.0), (64.0, 0.25)])
def test_yarn_divides_the_slow_pairs_and_keeps_the_fast(length, rotary, betas):
    fast, slow = betas
    factor = 4.0
    f, m = ttt.rope_frequencies(rotary, scaling="yarn", factor=factor, original_length=length, beta_fast=fast,
                                beta_slow=slow)
    plain = 10000.0 ** (-2.0 * np.arange(rotary // 2) / rotary)
    turns = length * plain / (2 * math.pi)
    ratio = f.double().numpy() / plain
    near = 2.0 ** -22  # the frequencies' rounding to fp32
    # (Pairs within 1e-9 of a bound may count on either side.)
    assert np.all(np.abs(ratio[turns < slow * (1 - 1e-9)] * factor - 1) <= near)
    assert np.all(np.abs(ratio[turns > fast * (1 + 1e-9)] - 1) <= near)
    assert np.all(ratio <= 1 + near) and np.all(ratio >= 1 / factor - near) and np.all(np.diff(ratio) <= near)
    assert m == 0.1 * math.log(factor) + 1.0
