"""Angles of the farthest positions.  A position of 31 bits times a frequency of 24 is a product of 55, more than
fp64 holds; the exact one, reduced to a turn with integers here, decides where it leaves a small angle, whose
sine shows an error of the angle in full."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import test_sequence_modeling_b200 as ttt
from linear_attn_helpers import D, U32

getcontext().prec = 60
TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")


def _reduced(position, mantissa):
    """position x mantissa 2^-23 less whole turns, within half a turn of zero."""
    a = Decimal(int(position) * int(mantissa)) / (1 << 23)
    return float(a - (a / TWO_PI).to_integral_value() * TWO_PI)


def _cases(seed=0):
    """Odd 24-bit mantissas for the 32 pairs (frequencies 1 to 2) and, for each, positions whose angle is
    within 0.02 of a whole turn: [(pair, position, angle)]."""
    rng = np.random.default_rng(seed)
    mantissas = rng.integers(1 << 22, 1 << 23, D // 2) * 2 + 1
    found = []
    for pair, m in enumerate(mantissas):
        p = rng.integers(1 << 30, 1 << 31, 4000) * rng.choice([-1, 1], 4000)
        near = np.remainder(p * (m / 2.0 ** 23) + np.pi, 2 * np.pi) - np.pi
        for at in p[np.abs(near) < 0.02][:12]:
            found.append((pair, int(at), _reduced(at, m)))
    return mantissas, found


def test_an_fp64_product_would_show():
    """The cases tell a rounded product from the exact one: its angle is off by more than the bound below."""
    mantissas, found = _cases()
    over = 0
    for pair, at, angle in found:
        a = float(at) * (int(mantissas[pair]) / 2.0 ** 23)
        r = float(Decimal(a) - (Decimal(a) / TWO_PI).to_integral_value() * TWO_PI)
        over += abs(r - angle) > 6 * U32 * abs(np.sin(angle)) + 4e-15
    assert len(found) > 300 and over > len(found) // 2


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_the_angle_is_the_exact_product(interleaved):
    mantissas, found = _cases()
    f = torch.from_numpy((mantissas / 2.0 ** 23).astype(np.float32)).cuda()
    x = torch.zeros(1, 1, len(found), D)
    x[..., 0::2 if interleaved else 1] = 1.0
    if not interleaved:
        x[..., D // 2:] = 0.0
    at = torch.tensor([[p for _, p, _ in found]], dtype=torch.int32).cuda()
    y, _ = ttt.ttt_rope(x.cuda(), None, ttt.Rope(f, interleaved=interleaved), positions=at)
    y = y.double().cpu().numpy()[0, 0]
    for t, (pair, at, angle) in enumerate(found):
        got = y[t, 2 * pair + 1] if interleaved else y[t, D // 2 + pair]
        # sincosf: within 2 units of the last place (4 half steps), the correction one more; the reduction in
        # fp64 leaves a few of its half steps of pi.  The pair (1, 0) adds none.
        assert abs(got - np.sin(angle)) <= 6 * U32 * abs(np.sin(angle)) + 4e-15, (pair, at)
