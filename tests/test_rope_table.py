"""The angles of rotary positions as the library lays them out (host code):
turns a position in 2^-64, against the formulas in 64 bits."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


def table(api, rd, base=10000.0, scaling="none", factor=1.0, context=0, low=0.0, high=0.0):
    turns, scale = (ctypes.c_uint64 * (rd // 2))(), ctypes.c_float()
    rc = api.lib.moe_rope_table(rd, base, api.ROPE_SCALINGS[scaling], factor, context, low, high, turns, ctypes.byref(scale))
    assert rc == api.OK
    return np.array(list(turns), np.float64) / 2.0 ** 64 * 2 * math.pi, scale.value


def close(got, want):
    """A few roundings of 64 bits: power, division, product. And half a unit
    of the fixed point, 2^-65 of a turn of 2 pi: a frequency of 2e-4 at 2^-49 of
    itself is below that."""
    assert (np.abs(got - want) <= 2.0 ** -49 * want + 2.0 ** -65 * 2 * math.pi).all()


@pytest.mark.parametrize("rd,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0), (512, 1.5)])
def test_frequencies(api, rd, base):
    f = base ** (-np.arange(0, rd, 2) / rd)
    got, scale = table(api, rd, base)
    close(got, f)
    assert scale == 1.0
    got, scale = table(api, rd, base, "linear", 8.0)
    close(got, f / 8)
    got, scale = table(api, rd, base, "ntk", 4.0)
    close(got, (base * 4.0 ** (rd / (rd - 2))) ** (-np.arange(0, rd, 2) / rd))
    assert scale == 1.0


@pytest.mark.parametrize("rd,base,factor,context", [(128, 10000.0, 4.0, 4096), (64, 1000000.0, 40.0, 32768), (32, 500000.0, 8.0, 8192)])
def test_frequencies_by_turns(api, rd, base, factor, context):
    f = base ** (-np.arange(0, rd, 2) / rd)
    turns = context * f / (2 * math.pi)
    # bands: all of the frequency from 4 turns on, a factor less below one
    got, scale = table(api, rd, base, "bands", factor, context)
    assert scale == 1.0
    close(got[turns >= 4], f[turns >= 4])
    close(got[turns <= 1], f[turns <= 1] / factor)
    between = (turns > 1) & (turns < 4)
    kept = (turns[between] - 1) / 3
    close(got[between], f[between] * kept + f[between] / factor * (1 - kept))
    # yarn: the ramp runs over the pairs' numbers between the borders, rounded outwards
    got, scale = table(api, rd, base, "yarn", factor, context)
    assert abs(scale - (0.1 * math.log(factor) + 1)) <= 2.0 ** -23
    i = np.arange(rd // 2)
    first = max(0, math.floor(rd * math.log(context / (32 * 2 * math.pi)) / (2 * math.log(base))))
    last = min(rd - 1, math.ceil(rd * math.log(context / (2 * math.pi)) / (2 * math.log(base))))
    assert (got[i <= first] == table(api, rd, base)[0][i <= first]).all()
    close(got[i >= last], f[i >= last] / factor)
    kept = np.clip(1 - (i - first) / (last - first), 0, 1)
    close(got, f * kept + f / factor * (1 - kept))
    # borders of one's own
    close(table(api, rd, base, "bands", factor, context, low=0.5, high=2.0)[0][turns >= 2], f[turns >= 2])


def test_any_frequencies(api):
    """Whole turns are dropped, a negative frequency turns the other way."""
    f = [math.pi, 2 * math.pi * 3.25, -2 * math.pi / 8, 0.0, 2 * math.pi]
    turns = (ctypes.c_uint64 * 5)()
    assert api.lib.moe_rope_turns((ctypes.c_double * 5)(*f), 5, turns) == api.OK
    # (3.25 turns in 64 bits are a multiple of 2^-51: 2^13 units)
    assert [turns[i] for i in (0, 2, 3, 4)] == [1 << 63, 7 << 61, 0, 0] and abs(turns[1] - (1 << 62)) <= 1 << 13
    assert api.lib.moe_rope_turns((ctypes.c_double * 1)(1e-12), 1, turns) == api.OK
    assert abs(turns[0] / 2.0 ** 64 * 2 * math.pi - 1e-12) < 2.0 ** -62


@pytest.mark.parametrize("over,code", [
    (dict(rd=8), "ESHAPE"), (dict(rd=24), "ESHAPE"), (dict(rd=528), "ESHAPE"), (dict(base=1.0), "EINVAL"), (dict(base=math.inf), "EINVAL"),
    (dict(base=math.nan), "EINVAL"), (dict(scaling=5), "EINVAL"), (dict(scaling=-1), "EINVAL"), (dict(factor=0.0), "EINVAL"),
    (dict(factor=math.nan), "EINVAL"), (dict(context=0), "EINVAL"), (dict(low=4.0, high=4.0), "EINVAL"), (dict(low=math.inf), "EINVAL"),
    (dict(turns=None), "EINVAL"), (dict(scale=None), "EINVAL")], ids=lambda v: str(v))
def test_refused_settings(api, over, code):
    a = dict(rd=64, base=10000.0, scaling=4, factor=8.0, context=8192, low=0.0, high=0.0, turns=(ctypes.c_uint64 * 300)(),
             scale=ctypes.byref(ctypes.c_float()))
    a.update(over)
    assert api.lib.moe_rope_table(*a.values()) == getattr(api, code)


def test_refused_frequencies(api):
    turns = (ctypes.c_uint64 * 2)()
    assert api.lib.moe_rope_turns((ctypes.c_double * 2)(1.0, math.nan), 2, turns) == api.EINVAL
    assert api.lib.moe_rope_turns(None, 2, turns) == api.EINVAL and api.lib.moe_rope_turns(None, -1, turns) == api.ESHAPE
    assert list(turns) == [0, 0]
    with pytest.raises(api.MoeError):
        api.Rope(64, scaling="other", device="cpu")
    with pytest.raises(api.MoeError):
        api.Rope(20, device="cpu")
