"""The oracle's angles at far positions against what holds for turns."""
import cmath
import math
import random

import pytest

import oracle
from oracle import step_oracle


def test_a_whole_turn():
    digits = "314159265358979323846264338327950288419716939937510582097494459230781640628620899862803"
    assert str(step_oracle._TURN // 2 * 10 ** 70 >> step_oracle._BITS) == digits[:71]


def test_near_positions_are_what_fp64_gives():
    for position in (0, 1, -1, 7, 1000, -4000):
        for freq in (0.0, 1.0, 0.125, 1e-4):
            a = oracle.angle_reference(position, freq)
            assert abs(a) <= math.pi
            assert cmath.isclose(cmath.rect(1, a), cmath.rect(1, position * freq), abs_tol=1e-12)


def test_far_positions_are_the_product_of_their_parts():
    """The turn of p + q is that of p and that of q, one after another."""
    r = random.Random(1)
    for _ in range(300):
        freq = float(r.choice((0.5, 1.0, 3.0, 511.0, 4096.0)) * (1 + r.getrandbits(23) * 2.0 ** -23))
        p, q = r.randint(-2 ** 31, 2 ** 31), r.randint(-2 ** 31, 2 ** 31)
        a, b, c = (cmath.rect(1, oracle.angle_reference(n, freq)) for n in (p, q, p + q))
        assert abs(a * b - c) <= 1e-14


@pytest.mark.parametrize("freq", [1.0, 511.0])
def test_a_rounded_turn_would_not_do(freq):
    """What fp64 alone gives at the end of 32 bits is off by more than fp32's step."""
    r = random.Random(2)
    worst = 0.0
    for _ in range(200):
        p = r.randint(2 ** 30, 2 ** 31)
        worst = max(worst, abs(cmath.rect(1, math.fmod(p * freq, 2 * math.pi)) - cmath.rect(1, oracle.angle_reference(p, freq))))
    assert worst > 2.0 ** -24
