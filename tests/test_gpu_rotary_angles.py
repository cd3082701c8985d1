"""Angles of rotary positions at high frequencies, against exact arithmetic: cosine
and sine within 2^-22, and their rounding to bf16."""
import math
from fractions import Fraction

import pytest
import torch

import segmented_dual_scale_amd as S
from gpu_common import DEV

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620,
                      10 ** 77)
PLACES = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 16777217, -99999989, 1000003, 3, 1, 0]


def check(freq, R):
    pos = torch.tensor(PLACES, device=DEV, dtype=torch.int32)[:, None].contiguous()
    x = torch.zeros(1, len(PLACES), 1, R, device=DEV, dtype=torch.bfloat16)
    x[..., ::2] = 1.0  # out = (cos, sin)
    out = S.segquant_qk_rotary(x, None, pos, freq.to(DEV), [R], S.SEGQ_ROTARY_PAIRS, norm=False)[0]
    for l, p in enumerate(PLACES):
        for i in range(R // 2):
            u = float(Fraction(p) * Fraction(float(freq[i])) % TWO_PI)
            for got, want in zip(out[0, l, 0, 2 * i:2 * i + 2].tolist(), (math.cos(u), math.sin(u))):
                assert abs(got - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -22, (p, float(freq[i]))


def test_angles_at_high_frequencies():
    freq = torch.tensor([1.0, 3.0, 1e3, -1e3, 1e6, 12345678.9, 1e9, -7e9, 1e12, 1e14, 2.0 ** 48,
                         0.1, 1e-5, 0.0, 5e7, 3e11], dtype=torch.float64)
    check(freq, 32)


@pytest.mark.parametrize("theta", [0.5, 1e-3, 1e-9, 1e-13])
def test_angles_of_a_theta_below_one(theta):
    """Its frequencies grow from pair to pair."""
    check(S.segquant_rotary_frequencies([64], theta), 64)
