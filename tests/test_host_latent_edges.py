"""Host parts of the rotary positions where they can go wrong, without a GPU."""

import ctypes as C
from fractions import Fraction

import numpy as np

from prefix_shared_kv_token_gb300 import _lib

lib = _lib.lib


def arctan_inverse(n, bits):
    """arctan(1 / n) in 2^-bits, by its series."""
    total = term = (1 << bits) // n
    k = 1
    while term:
        term //= -n * n
        k += 2
        total += term // k
    return total


def phases(freq):
    f, out = np.ascontiguousarray(freq, np.float64), np.zeros(len(freq), np.uint64)
    at = lambda a: a.ctypes.data_as(C.c_void_p)  # noqa: E731
    assert lib.pkv_rope_phases(at(f), len(f), at(out)) == 0
    return [int(x) for x in out]


def test_phases_of_any_sign_are_a_doubles():
    """Against 1 / 2 pi in 1,300 bits (Machin's formula).  The division by 2 pi is off by 2^-53 of its result, the 2 pi it
    divides by by 2^-54.5 of itself, the phase by half a unit: 2^-52 |f| / 2 pi turns and that half."""
    bits = 1300
    pi = Fraction(4 * (4 * arctan_inverse(5, bits) - arctan_inverse(239, bits)), 1 << bits)
    rng = np.random.default_rng(1)
    freq = np.concatenate([[1.0, 2.0, 100.0, 1000.5, 1e-4, 1e-9, 0.01, 3.0, 1e12, 5e-324], 500000.0 ** (-np.arange(64) / 64),
                           10.0 ** rng.uniform(-12, 6, 200)])
    plus, minus = phases(freq), phases(-freq)
    for f, a, b in zip(freq, plus, minus):
        turns = Fraction(float(f)) / (2 * pi)
        off = (Fraction(a, 1 << 64) - turns + Fraction(1, 2)) % 1 - Fraction(1, 2)
        assert abs(off) <= turns / (1 << 52) + Fraction(1, 1 << 65), f
        assert (a + b) % (1 << 64) == 0, f         # turns back by as much
