"""Whole numbers beyond 32 bits: the binding refuses them instead of letting
their lower 32 bits through (this suite also runs without a GPU)."""
import pytest
import torch

from test_abi_cache8 import t
from test_abi_paged import Calls
from test_abi_tree import attention_call

BEYOND = [1 << 31, (1 << 32) + 8192, -(1 << 31) - 1, 1 << 64]


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


@pytest.fixture
def calls(api, monkeypatch):
    calls = Calls(api.lib)
    monkeypatch.setattr(api, "lib", calls)
    monkeypatch.setattr(api, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    return calls


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("window", BEYOND)
def test_windows(api, calls, codes, window):
    fn, a = attention_call(api, codes)
    a["tree_masks"] = None
    with pytest.raises(api.MoeError):
        fn(**a, window=window)
    assert not calls.made
    fn(**a, window=(1 << 31) - 1)
    assert len(calls.made) == 1


@pytest.mark.parametrize("block_size", BEYOND)
def test_block_sizes(api, calls, block_size):
    i = torch.int32
    a = dict(ctx_lens=t(i, 2), new_lens=t(i, 2), free_list=t(i, 8), block_tables=t(i, 2, 4), q_start=t(i, 3), seq_lens=t(i, 2),
             slot_map=t(i, 5), taken=t(i, 1), ws=t(torch.uint8, 1024))
    with pytest.raises(api.MoeError):
        api.paged_plan(block_size=block_size, **a)
    assert not calls.made


@pytest.mark.parametrize("number", BEYOND)
def test_angles(api, number):
    with pytest.raises(api.MoeError):
        api.Rope(64, scaling="yarn", factor=4.0, context=number, device="cpu")
    with pytest.raises(api.MoeError):
        api.Rope(number + 64, device="cpu")
    with pytest.raises(api.MoeError):
        api.Rope(1024, device="cpu")
