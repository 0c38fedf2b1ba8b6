"""The turns of a rotation against decimal arithmetic of 80 digits: every bit of the 64 counts, since a position multiplies
them, and frequencies that no turn can stand for are refused."""
import ctypes
import math
from decimal import Decimal as D, getcontext

import numpy as np
import pytest

getcontext().prec = 80
# 2 pi by Machin's formula
def _atan_inv(n):
    x, total, k = D(1) / n, D(0), 0
    term = x
    while abs(term) > D(10) ** -85:
        total += term / (2 * k + 1) * (-1) ** k
        term /= n * n
        k += 1
    return total


TAU = 8 * (4 * _atan_inv(5) - _atan_inv(239))


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_group_quantized_gb300 as fg
    return fg


def _fractions(rot, scaling, base, factor, context, low, high):
    """theta_i / 2 pi, one by one (the numbers given are doubles, exactly)."""
    base, factor, context, low, high = (D(x) for x in (base, factor, context, low, high))
    if scaling == "base":
        base = (base.ln() + factor.ln() * rot / (rot - 2)).exp()
    for i in range(rot // 2):
        t = (base.ln() * (-2 * i) / rot).exp()
        if scaling == "linear":
            t /= factor
        elif scaling == "bands":
            share = min(D(1), max(D(0), (context * t / TAU - low) / (high - low)))
            t = share * t + (1 - share) * t / factor
        elif scaling == "ramp":
            def number(turns):
                return rot * (context / (TAU * turns)).ln() / (2 * base.ln())
            a, z = max(0, math.floor(number(high))), min(rot - 1, math.ceil(number(low)))
            share = min(D(1), max(D(0), D(i - a) / max(D(z - a), D(0.001))))
            t = (1 - share) * t + share * t / factor
        yield t / TAU


NUMBERS = [(10000.0, 8.0, 4096.0, 1.0, 4.0), (5e5, 32.0, 8192.0, 1.0, 32.0), (1e6, 40.0, 32768.0, 0.7, 31.3),
           (10000.0, 1.0, 100.0, 0.5, 2.0), (1.5, 3.0, 64.0, 1.0, 2.0), (1e30, 1.1, 1e9, 1e-3, 1e3)]


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "bands", "ramp"])
@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128])
def test_every_bit_of_the_turns(fg, scaling, rot):
    if scaling == "base" and rot == 2:
        pytest.skip("refused: a rotation of two dims has no other base")
    for numbers in NUMBERS:
        turns, _ = fg.fg_rotary_turns(rot, fg._SCALINGS[scaling], *numbers)
        got = turns.numpy().view(np.uint64)
        for g, part in zip(got, _fractions(rot, scaling, *numbers)):
            off = (D(int(g)) - part * 2 ** 64) % 2 ** 64
            # rounded to the nearest: half a unit, and 2^-10 of one for what 100 bits leave of numbers up to 2^26 turns
            assert min(off, 2 ** 64 - off) <= D("0.501"), (numbers, float(off))


@pytest.mark.parametrize("base", [10000.0, 5e5])
@pytest.mark.parametrize("pos", [200_000, 2 ** 24 + 1, 2 ** 31 - 1, -(2 ** 31)])
def test_angles_of_far_positions(fg, base, pos):
    """A position times the turns is its angle to half a unit of 2^-64 for each of its steps: 2^-34 turns at the farthest."""
    turns, _ = fg.fg_rotary_turns(128, base=base)
    for g, part in zip(turns.numpy().view(np.uint64), _fractions(128, "plain", base, 1, 1, 1, 2)):
        got, want = D(pos * int(g) % 2 ** 64) / 2 ** 64, part * pos % 1
        off = (got - want) % 1
        assert min(off, 1 - off) <= D(abs(pos)) * D("0.501") / 2 ** 64


def test_frequencies_that_no_turn_stands_for(fg):
    """Numbers that are fine one by one, whose frequencies (or base) are not numbers or 2^32 turns and more."""
    t = (ctypes.c_uint64 * 64)(*[7] * 64)
    s = ctypes.c_float(7.0)

    def turns(kind, base=1e4, factor=2.0, context=100.0, low=1.0, high=2.0, rot=64):
        return fg.lib.fg_rotary_turns(rot, kind, base, factor, context, low, high, t, ctypes.byref(s))

    assert turns(1, factor=1e-320) == 1 and turns(1, factor=1e-300) == 1 and turns(1, factor=1e-12) == 1
    assert turns(2, factor=1e-300) == 1 and turns(2, factor=1e300, rot=4) == 1 and turns(2, base=1e300, factor=1e300) == 1
    assert turns(3, factor=1e-320) == 1 and turns(3, factor=1e-300) == 1
    assert list(t) == [7] * 64 and s.value == 7.0            # nothing is written
    assert turns(1, factor=1e-9) == 0 and turns(1, factor=1e300) == 0 and turns(0, base=1e308) == 0
