"""Turns per position of rotary frequencies (swa_rotary_turns) against integers: 2 pi to 600 bits,
so that every one of the 64 bits is checked."""
import ctypes
from fractions import Fraction

import pytest

from sliding_window_gqa_prep_gb300 import _abi
import sliding_window_gqa_prep_gb300 as swa

BITS = 600


def _arctan_inv(x):
    """2^BITS arctan(1 / x) by its series."""
    term = (1 << BITS) // x
    total, n, sign = term, 3, -1
    while term:
        term //= x * x
        total += sign * (term // n)
        n, sign = n + 2, -sign
    return total


PI = Fraction(4 * (4 * _arctan_inv(5) - _arctan_inv(239)), 1 << BITS)      # off by less than 2^-590

SCHEDULES = [
    dict(rot=64, theta=10000.0), dict(rot=256, theta=10000.0), dict(rot=2, theta=500000.0), dict(rot=1024, theta=1e8),
    dict(rot=20, theta=1e6, schedule="linear", factor=4.0), dict(rot=128, theta=10000.0, schedule="base", factor=8.0),
    dict(rot=128, theta=10000.0, schedule="parts", factor=16.0, orig_len=4096),
    dict(rot=64, theta=0.5),                       # frequencies above 1, up to 2
    dict(rot=128, theta=1e-19),                    # up to 2^62: most of the bits drop out
    dict(rot=64, theta=1e300),                     # down to 2^-965: zeros
]


@pytest.mark.parametrize("kw", SCHEDULES)
def test_every_bit_of_the_turns(kw):
    f = swa.rotary_freqs(**kw).tolist()
    t = swa.rotary_turns(device="cpu", **kw).tolist()
    for x, got in zip(f, t):
        turn = Fraction(x) / (2 * PI)
        assert got % (1 << 64) == (turn - (turn.numerator // turn.denominator)) * (1 << 64) // 1
        # and what that makes of far positions: 2^-33 turns
        for pos in (1, 77777, (1 << 31) - 1, -(1 << 31)):
            want = pos * turn % 1
            d = abs(Fraction(pos * got % (1 << 64), 1 << 64) - want)
            assert min(d, 1 - d) <= Fraction(1, 1 << 33)


def test_frequencies_past_the_range_are_refused():
    lib = _abi.load()
    s = _abi.RotarySchedule()
    s.kind, s.rot, s.theta, s.factor = 0, 4, 2.0 ** -126, 1.0                # 1 and 2^63
    f, t = (ctypes.c_double * 2)(), (ctypes.c_uint64 * 2)()
    assert lib.swa_rotary_turns(ctypes.byref(s), f, t) == _abi.SWA_OK and f[1] == 2.0 ** 63
    s.theta = 2.0 ** -128                                                   # 2^64
    f[0] = t[0] = 7
    assert lib.swa_rotary_turns(ctypes.byref(s), f, t) == _abi.SWA_E_SHAPE
    assert f[0] == 7 and t[0] == 7
