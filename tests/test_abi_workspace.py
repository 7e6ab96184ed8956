"""The places of a workspace that the attentions over both kinds of cache share
(this suite also runs without a GPU)."""
import ctypes

import pytest

from test_abi_cache8 import cache8
from test_abi_paged import cache

COUNTERS, ROWS = 256, 32  # CTAs of a launch at the most, rows of an item


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


@pytest.mark.parametrize("d", [64, 128])
def test_parts_lie_behind_all_counters(api, d):
    """The attention over 16 bits keeps three counters a CTA behind the control
    block and needs them zero: the parts of the one over codes, two of 32 rows a
    CTA, begin behind them."""
    c = cache8(api, head_dim=d, k_head_stride=d, v_head_stride=d, k_token_stride=2 * d, v_token_stride=2 * d)
    n = api.lib.moe_paged_attention8_workspace_bytes(8, ctypes.byref(c))
    assert n - 2 * COUNTERS * ROWS * (d + 2) * 4 == api.PAGED_WORKSPACE_BYTES + 3 * 4 * COUNTERS


def test_a_workspace_for_16_bits_is_the_larger_one(api):
    c8 = cache8(api, head_dim=128, k_head_stride=128, v_head_stride=128, k_token_stride=256, v_token_stride=256)
    least = min(api.lib.moe_paged_attention_workspace_bytes(8, ctypes.byref(cache(api, head_dim=d, k_head_stride=d, v_head_stride=d))) for d in (64, 128))
    assert 0 < api.lib.moe_paged_attention8_workspace_bytes(8, ctypes.byref(c8)) <= least
