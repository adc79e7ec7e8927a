"""Host parts of the rotary positions where they can go wrong, without a GPU."""

import ctypes as C
from fractions import Fraction

import numpy as np
import pytest

import prefix_shared_kv_token_gb300 as pkv
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


def test_zero_padded_refusals():
    P = 0x10000                                    # stands for a device address (never read)

    def call(out=P, tok=1024, head=128, heads=8, dim=128, loc=P, n=4):
        return lib.pkv_zero_padded(out, tok, head, heads, dim, loc, n, None)

    for kw in (dict(out=None), dict(out=P + 8), dict(tok=0), dict(tok=1020), dict(head=0), dict(head=4), dict(heads=-1), dict(dim=0),
               dict(loc=None), dict(n=-1)):
        assert call(**kw) == -1, kw
    for kw in (dict(dim=132), dict(dim=520), dict(heads=65537), dict(n=1 << 40)):
        assert call(**kw) == -2, kw
    assert call(n=0, out=None) == 0 and call(heads=0, out=None) == 0


@pytest.mark.parametrize("original,fast,slow", [(4096, 32, 1), (6, 32, 1), (3, 32, 1), (100, 64, 32), (100, 20, 15), (10 ** 9, 32, 1)])
def test_yarn_keeps_fast_pairs_and_divides_slow_ones(original, fast, slow):
    """Also where no pair is fast, or all are, within the original context."""
    plain = pkv.Rope(64, device="cpu").inv_freq
    ratio = pkv.Rope(64, scaling=dict(kind="yarn", factor=8, original=original, beta_fast=fast, beta_slow=slow), device="cpu").inv_freq / plain
    turns = original * plain / (2 * np.pi)
    # the ramp's ends are whole pairs, one further out at most
    step = 10000.0 ** (1 / 32)
    assert np.allclose(ratio[turns > fast * step], 1.0, rtol=1e-15) and np.allclose(ratio[turns < slow / step], 1 / 8, rtol=1e-15)
    assert np.all((ratio <= 1 + 1e-15) & (ratio >= 1 / 8 - 1e-15) & (np.diff(ratio, prepend=1.0) <= 1e-15))
    if turns.max() < slow:
        assert np.allclose(ratio, 1 / 8, rtol=1e-15)
