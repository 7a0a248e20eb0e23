"""Frequency tables of rotary positions (no GPU needed)."""
import math

import pytest

from resident_expert_routed_gb300.rotary import rotary_frequencies, rotary_magnitude, rotary_turns


def test_turns_hold_the_frequencies():
    f = rotary_frequencies(128)
    t = rotary_turns(f, device="cpu").tolist()
    assert len(f) == len(t) == 64 and f[0] == 1.0
    for x, n in zip(f, t):
        # a quotient in 64 bits is off by 2^-53 of itself, the whole number by half of one
        assert abs(n % 2 ** 64 - x / (2 * math.pi) * 2.0 ** 64) <= 0.5 + 2.0 ** -51 * x * 2.0 ** 64


def test_whole_turns_are_none_and_signs_wrap():
    t = rotary_turns([2 * math.pi, -1.0, 1.0, 4.0], device="cpu").tolist()
    assert abs(t[0]) < 2 ** 13 and t[1] == -t[2]                    # (2 pi rounded to 64 bits is not 2 pi)
    assert t[3] < 0                                                  # above half a turn: the upper bit


def test_rules():
    f = rotary_frequencies(64)
    assert rotary_frequencies(64, stretch=4.0) == [x / 4.0 for x in f]
    g = rotary_frequencies(64, stretch=4.0, rule="base")
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 4.0, rel_tol=1e-12) and all(a >= b for a, b in zip(f, g))
    r = rotary_frequencies(64, stretch=4.0, rule="ramp", trained=4096)
    assert r[0] == f[0] and r[-1] == f[-1] / 4.0 and all(x / 4.0 <= y <= x for x, y in zip(f, r))
    assert rotary_magnitude(1.0) == 1.0 and rotary_magnitude(math.e) == pytest.approx(1.1)


@pytest.mark.parametrize("kw", [dict(turned=0), dict(turned=7), dict(turned=8, base=1.0), dict(turned=8, stretch=0.5),
                                dict(turned=8, rule="other"), dict(turned=2, rule="base", stretch=2.0), dict(turned=8, fast=1.0)])
def test_refusals(kw):
    with pytest.raises(ValueError):
        rotary_frequencies(**kw)
