"""Frequency tables of rotary positions for ``moe_qk_rotate``.

``rotary_frequencies`` gives the radians a position of each pair, as Python floats (64 bits); ``rotary_turns`` the same as
whole numbers of 2^-64 turns, which the kernel multiplies by the position exactly.
"""
from __future__ import annotations

import math
from fractions import Fraction

import torch

# 1 / (2 pi) to 2^-120 (pi to 40 digits)
_PI = Fraction(3141592653589793238462643383279502884197, 10 ** 39)
_TURN = 1 / (2 * _PI)


def rotary_frequencies(turned: int, base: float = 10000.0, stretch: float = 1.0, rule: str = "linear", trained: int = 4096,
                       fast: float = 32.0, slow: float = 1.0) -> list[float]:
    """Radians a position of the `turned` / 2 pairs of a head: base^(-2 i / turned).

    stretch > 1 reaches that many times the trained length. rule "linear": every frequency divided by it. "base": the
    base raised so that the slowest frequency is divided by it and the fastest stays. "ramp": pairs that turn less than
    `slow` times in the trained length are divided, those of more than `fast` turns stay, between them a ramp that is linear
    in the turns (the factor for the turned values that goes with it is ``rotary_magnitude``). Checkpoints whose ramp is
    linear in the pair's index have other frequencies between the two: ``rotary_turns`` takes any list."""
    if turned < 2 or turned % 2 or not base > 1.0 or not stretch >= 1.0 or rule not in ("linear", "base", "ramp") or not fast > slow:
        raise ValueError("turned: an even number from 2; base > 1; stretch >= 1; rule linear, base or ramp; fast > slow")
    if rule == "base" and stretch > 1.0:
        if turned < 4:
            raise ValueError("rule base: two pairs at least")
        base *= stretch ** (turned / (turned - 2))
    f = [base ** (-2.0 * i / turned) for i in range(turned // 2)]
    if rule == "linear":
        return [x / stretch for x in f]
    if rule == "base":
        return f
    keep = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
    return [x * k + x / stretch * (1.0 - k) for x, k in zip(f, keep)]


def rotary_magnitude(stretch: float) -> float:
    """The factor of the turned values that goes with rule "ramp": 0.1 ln(stretch) + 1."""
    return 0.1 * math.log(stretch) + 1.0


def rotary_turns(frequencies: list[float], device="cuda") -> torch.Tensor:
    """int64 [pairs]: the frequencies as whole numbers of 2^-64 turns (modulo 2^64), for ``moe_qk_rotate``."""
    whole = [round(Fraction(float(f)) * _TURN * 2 ** 64) % 2 ** 64 for f in frequencies]
    return torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in whole], dtype=torch.int64, device=device)
