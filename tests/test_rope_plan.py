"""The plan of the rotation: what it refuses, with its outputs left as they were."""
import ctypes

import numpy as np
import pytest

import int8_kv_cache_quant_gb300 as k

KINDS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4, "divisors": 5}


def plan(r, base, kind="none", factor=1.0, original_len=0.0, low=1.0, high=32.0, divisors=None):
    div = (ctypes.c_double * len(divisors))(*divisors) if divisors else None
    z = k.kvq._RopeScaling(KINDS[kind], factor, original_len, low, high,
                           ctypes.cast(div, ctypes.POINTER(ctypes.c_double)) if div else None)
    out = np.full(r // 2, 7, np.uint64)
    af = ctypes.c_float(5.0)
    st = k.lib().kvq_rope_phases(r, base, ctypes.byref(z), out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), ctypes.byref(af))
    return st, out, af.value


@pytest.mark.parametrize("kw", [
    dict(r=128, base=5e-324), dict(r=8, base=1e4, kind="linear", factor=1e-310), dict(r=4, base=1e4, kind="ntk", factor=1e-300),
    dict(r=8, base=1e4, kind="yarn", factor=1e-310, original_len=4096.0), dict(r=8, base=1e4, kind="bands", factor=1e-310, original_len=64.0),
    dict(r=8, base=1e4, kind="divisors", divisors=[1.0, 2.0, 3.0, 1e-320]),
    dict(r=8, base=1e4, kind="divisors", divisors=[1.0, 2.0, 3.0, 0.0]),
    dict(r=8, base=1e4, kind="divisors", divisors=[1.0, 2.0, 3.0, float("nan")])])
def test_a_frequency_that_is_no_number_is_refused_and_nothing_is_written(kw):
    st, out, af = plan(**kw)
    assert st == 1 and (out == 7).all() and af == 5.0


@pytest.mark.parametrize("kw", [dict(r=128, base=1e-300), dict(r=8, base=1.7e308), dict(r=8, base=1e4, kind="linear", factor=1e300),
                                dict(r=8, base=1e4, kind="divisors", divisors=[1.0, 2.0, 3.0, float("inf")])])
def test_frequencies_at_the_ends_of_a_double_are_taken(kw):
    st, out, af = plan(**kw)
    assert st == 0 and not (out == 7).any() and af == 1.0


@pytest.mark.parametrize("base,r", [(500.0, 6), (1e4, 64), (1e4, 256), (1e6, 128), (1e7, 1024)])
def test_angles_of_far_positions_against_the_frequencies(base, r):
    """At position 2^31, against 50 digits.  The plan rounds in double precision: the exponent 2j / r (2^-53 relative,
    which moves base^-x by at most x ln(base) base^-x <= 1/e of that), the power (an ulp, 2^-52 relative), 2 pi and the
    division by it (2^-53 each), all on a frequency of at most 1; then half of 2^-64 turns.  That is 4.4 times 2^-53 in
    the angle per position."""
    from decimal import Decimal, getcontext
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    st, out, _ = plan(r, base)
    assert st == 0
    for j in range(r // 2):
        turns = Decimal(base) ** (Decimal(-2 * j) / Decimal(r)) / two_pi
        err = abs(Decimal(int(out[j])) / 2 ** 64 - turns % 1) * two_pi * 2 ** 31
        assert err <= Decimal(4.4 * 2.0 ** -22 + 2.0 ** -31), (j, err)
