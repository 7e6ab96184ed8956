"""The turns of the tables of rotary positions to their last unit, 2^-64 of a
turn, against the formulas in 90 digits: what a turn is off by, a position
multiplies by up to 2^31."""
import ctypes
from decimal import ROUND_FLOOR, Decimal, getcontext

import pytest

getcontext().prec = 90


def pi():
    """16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan(n):
        s, term, k = Decimal(0), Decimal(1) / n, 1
        while abs(term) > Decimal(10) ** -95:
            s += term / k if k % 4 == 1 else -term / k
            term, k = term / (n * n), k + 2
        return s
    return 16 * arctan(5) - 4 * arctan(239)


TWO_PI = 2 * pi()


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


def frequencies(rd, base, scaling, factor, context, low, high):
    base, factor, n = Decimal(base), Decimal(factor), Decimal(rd)
    if scaling == "ntk":
        base *= factor ** (n / (n - 2))
    f = [base ** (-2 * Decimal(i) / n) for i in range(rd // 2)]
    if scaling in ("none", "ntk"):
        return f
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling == "bands":
        kept = [(context * x / TWO_PI - low) / (high - low) for x in f]
    else:
        at = [n * (context / (turns * TWO_PI)).ln() / (2 * base.ln()) for turns in (high, low)]
        first = max(at[0].to_integral_value(ROUND_FLOOR), 0)
        last = min(-(-at[1]).to_integral_value(ROUND_FLOOR), rd - 1)
        kept = [1 - (i - first) / (last - first) for i in range(rd // 2)]
    kept = [min(max(k, Decimal(0)), Decimal(1)) for k in kept]
    return [x * k + x / factor * (1 - k) for x, k in zip(f, kept)]


@pytest.mark.parametrize("rd,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0), (128, 1.0e6), (512, 1.5), (96, 3.0e7), (32, 1.0000001)])
@pytest.mark.parametrize("scaling,factor,context,low,high", [
    ("none", 0.0, 0, 0, 0), ("linear", 8.0, 0, 0, 0), ("linear", 0.3, 0, 0, 0), ("linear", 1e-9, 0, 0, 0), ("ntk", 4.0, 0, 0, 0), ("ntk", 1.7, 0, 0, 0),
    ("yarn", 40.0, 4096, 0, 0), ("yarn", 4.0, 32768, 0, 0), ("bands", 8.0, 8192, 0, 0), ("bands", 3.3, 5000, 0.7, 2.9)])
def test_turns_to_the_last_unit(api, rd, base, scaling, factor, context, low, high):
    if scaling == "yarn" and base < 2:
        pytest.skip("both borders beyond the pairs")
    turns, scale = (ctypes.c_uint64 * (rd // 2))(), ctypes.c_float()
    assert api.lib.moe_rope_table(rd, base, api.ROPE_SCALINGS[scaling], factor, context, low, high, turns, ctypes.byref(scale)) == api.OK
    borders = Decimal(low or 1), Decimal(high or (32 if scaling == "yarn" else 4))
    for t, f in zip(turns, frequencies(rd, base, scaling, factor, context, *borders)):
        want = f / TWO_PI % 1 * 2 ** 64
        off = abs(Decimal(t) - want)
        # (half a unit of rounding, and what some 106 bits leave of frequencies up to 2^30)
        assert min(off, 2 ** 64 - off) < 1


def test_angles_far_out(api):
    """At position 2^31 - 1 a pair's angle, in turns of 2^-32."""
    turns, scale, p = (ctypes.c_uint64 * 64)(), ctypes.c_float(), (1 << 31) - 1
    assert api.lib.moe_rope_table(128, 500000.0, 0, 1.0, 0, 0.0, 0.0, turns, ctypes.byref(scale)) == api.OK
    for t, f in zip(turns, frequencies(128, 500000.0, "none", 1.0, 0, 0, 0)):
        off = abs(Decimal(p * t % 2 ** 64 >> 32) - p * f / TWO_PI % 1 * 2 ** 32)
        assert min(off, 2 ** 32 - off) <= Decimal("1.5")


def test_turns_of_frequencies_in_64_bits(api):
    """As good as a division of 64 bits: 2^-52 of the turns (pi is half a turn)."""
    f = [1.0, 0.3, 1e-5, 123.456, -2.5, 3.141592653589793]
    turns = (ctypes.c_uint64 * len(f))()
    assert api.lib.moe_rope_turns((ctypes.c_double * len(f))(*f), len(f), turns) == api.OK
    for t, x in zip(turns, f):
        want = Decimal(x) / TWO_PI
        off = (Decimal(t) / 2 ** 64 - want) % 1
        assert min(off, 1 - off) <= abs(want) * Decimal(2) ** -52 + Decimal(2) ** -64
    assert turns[5] == 1 << 63


@pytest.mark.parametrize("scaling,base,factor,context", [
    ("linear", 10000.0, 1e-310, 0), ("yarn", 10000.0, 1e-310, 4096), ("bands", 10000.0, 5e-324, 4096), ("ntk", 10000.0, 5e-324, 0),
    ("ntk", 1e300, 1e300, 0), ("ntk", 1e-3 + 1, 5e-324, 0)])
def test_frequencies_that_overflow_are_refused(api, scaling, base, factor, context):
    turns, scale = (ctypes.c_uint64 * 32)(*([7] * 32)), ctypes.c_float(3.0)
    assert api.lib.moe_rope_table(64, base, api.ROPE_SCALINGS[scaling], factor, context, 0.0, 0.0, turns, ctypes.byref(scale)) == api.EINVAL
    assert list(turns) == [7] * 32 and scale.value == 3.0


@pytest.mark.parametrize("scaling,base,factor", [("none", 1.7e308, 0.0), ("linear", 1e4, 1e-200), ("ntk", 1e4, 1e-20), ("ntk", 10.0, 1e290),
                                                 ("ntk", 1e4, 1e-310)])  # (1e-310^(32/31) is above 0, and 1e316^(31/32) finite)
def test_far_settings_are_taken(api, scaling, base, factor):
    """The pairs whose frequency is small enough for 64 bits to hold its turns."""
    turns, scale = (ctypes.c_uint64 * 32)(), ctypes.c_float()
    assert api.lib.moe_rope_table(64, base, api.ROPE_SCALINGS[scaling], factor, 0, 0.0, 0.0, turns, ctypes.byref(scale)) == api.OK
    for t, f in zip(turns, frequencies(64, base, scaling, factor, 0, 0, 0)):
        if f < 2 ** 20:
            off = (Decimal(t) / 2 ** 64 - f / TWO_PI) % 1
            assert min(off, 1 - off) <= f * Decimal(2) ** -45 + Decimal(2) ** -63
