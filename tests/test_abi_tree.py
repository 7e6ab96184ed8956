"""Host-side refusals of trees of drafted tokens and of attention over the cache
of 8-bit values: every case returns its code before any launch (this suite also
runs without a GPU)."""
import ctypes

import pytest
import torch

from test_abi_cache8 import NAMES, binding_call, cache8, call, t
from test_abi_paged import BAD_CACHES, F, Calls, OnGpu, OnHost, OnOtherGpu, cache


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


@pytest.fixture
def calls(api, monkeypatch):
    calls = Calls(api.lib)
    calls.moe_rope_table = api.lib.moe_rope_table  # host code
    monkeypatch.setattr(api, "lib", calls)
    monkeypatch.setattr(api, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    return calls


ARGS = dict(q=F, qt=512, qh=64, T=4, heads=8, tables=F, width=8, q_start=F, seq=F, masks=F, B=2, scale=0.0, out=F, lse=F, ws=F, ws_bytes=1 << 30)


def attend(api, c=None, **over):
    a = {**ARGS, **over}
    return api.lib.moe_paged_tree_attention(a["q"], a["qt"], a["qh"], a["T"], a["heads"], ctypes.byref(c or cache(api)), a["tables"],
                                            a["width"], a["q_start"], a["seq"], a["masks"], a["B"], a["scale"], a["out"], a["lse"], a["ws"],
                                            a["ws_bytes"], None)


def attend8(api, c=None, dtype=0, window=0, **over):
    a = {**ARGS, **over}
    return api.lib.moe_paged_attention8(a["q"], a["qt"], a["qh"], a["T"], a["heads"], dtype, ctypes.byref(c or cache8(api)), a["tables"],
                                        a["width"], a["q_start"], a["seq"], a["masks"], a["B"], a["scale"], window, a["out"], a["lse"],
                                        a["ws"], a["ws_bytes"], None)


BOTH = [
    (dict(heads=7), "ESHAPE"), (dict(heads=0), "ESHAPE"), (dict(heads=128), "ESHAPE"), (dict(T=-1), "ESHAPE"),
    (dict(T=1 << 30), "ESHAPE"), (dict(B=0), "ESHAPE"), (dict(B=4097), "ESHAPE"), (dict(width=0), "ESHAPE"),
    (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(q=None), "EINVAL"), (dict(out=None), "EINVAL"),
    (dict(tables=None), "EINVAL"), (dict(q_start=None), "EINVAL"), (dict(seq=None), "EINVAL"), (dict(q=F + 8), "EALIGN"),
    (dict(out=F + 4), "EALIGN"), (dict(lse=F + 2), "EALIGN"), (dict(tables=F + 1), "EALIGN"), (dict(masks=F + 4), "EALIGN"),
    (dict(qt=516), "ESHAPE"), (dict(qh=-64), "ESHAPE"), (dict(ws=None), "EWORKSPACE"), (dict(ws=F + 4), "EALIGN"),
    (dict(ws_bytes=1024), "EWORKSPACE")]


@pytest.mark.parametrize("over,code", BOTH + [(dict(masks=None), "EINVAL")], ids=lambda v: str(v))
def test_tree_attention(api, over, code):
    assert attend(api, **over) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("over,code", BAD_CACHES, ids=lambda v: str(v))
def test_tree_attention_caches(api, over, code):
    assert attend(api, cache(api, **over)) == getattr(api, code)


@pytest.mark.parametrize("over,code", BOTH + [(dict(dtype=2), "ESHAPE"), (dict(window=-1, masks=None), "ESHAPE"), (dict(window=5), "ESHAPE")],
                         ids=lambda v: str(v))
def test_attention8(api, over, code):
    assert attend8(api, **over) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("over,code", [
    (dict(k=None), "EINVAL"), (dict(k_scale=None), "EINVAL"), (dict(head_dim=96), "ESHAPE"), (dict(block_size=24), "ESHAPE"),
    (dict(kv_heads=257), "ESHAPE"), (dict(v_token_stride=72), "ESHAPE"), (dict(v=F + 8), "EALIGN")], ids=lambda v: str(v))
def test_attention8_caches(api, over, code):
    c = cache8(api, **over)
    assert attend8(api, c) == getattr(api, code)
    assert api.lib.moe_paged_attention8_workspace_bytes(8, ctypes.byref(c)) == 0


def test_workspace_bytes(api):
    n = api.lib.moe_paged_attention8_workspace_bytes
    c = ctypes.byref(cache8(api))
    assert n(8, c) > api.PAGED_WORKSPACE_BYTES and n(7, c) == n(0, c) == n(66, c) == 0
    assert attend8(api, ws_bytes=n(8, c) - 1) == api.EWORKSPACE


def test_nothing_to_do(api):
    assert attend(api, T=0, q=None, out=None) == attend8(api, T=0, q=None, out=None) == api.OK
    assert api.lib.moe_tree_plan(None, None, None, 1, 0, None, None, None, 0, None) == api.OK
    # (tensors of no tokens have no address)
    for name in ("moe_rope", "moe_paged_rope_append", "moe_paged_rope_append8"):
        assert call(api, name, T=0, q=None, qo=None, k=None, ko=None, v=None, slots=None, positions=None, ws=None) == api.OK


@pytest.mark.parametrize("at,value,code", [
    (0, None, "EINVAL"), (1, None, "EINVAL"), (2, None, "EINVAL"), (3, 0, "ESHAPE"), (3, 4097, "ESHAPE"), (4, -1, "ESHAPE"),
    (5, None, "EINVAL"), (5, F, "EINVAL"), (6, F + 4096, "EINVAL"), (0, F + 2, "EALIGN"), (5, F + 12292, "EALIGN"), (6, F + 1, "EALIGN"),
    (7, None, "EWORKSPACE"), (7, F + 8, "EALIGN"), (8, 1023, "EWORKSPACE")])
def test_tree_plan(api, at, value, code):
    args = [F, F + 4096, F + 8192, 2, 8, F + 12288, F + 16384, F + 20480, 1024, None]
    args[at] = value
    assert api.lib.moe_tree_plan(*args) == getattr(api, code)
    assert api.last_launch_count() == 0


def attention_call(api, codes):
    i, f, b, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    a = dict(q=t(b, 3, 4, 64), block_tables=t(i, 2, 4), q_start=t(i, 3), seq_lens=t(i, 2), out=t(b, 3, 4, 64), ws=t(u8, 1024), lse=t(f, 3, 4),
             tree_masks=t(torch.int64, 3), ck=t(u8 if codes else b, 8, 16, 2, 64), cv=t(u8 if codes else b, 8, 16, 2, 64))
    if codes:
        a.update(ks=t(u8, 8, 2, 16), vs=t(u8, 8, 2, 16))

    def held(ck, cv, ks=None, vs=None):
        return api.KvCache8(ck, cv, ks, vs) if codes else api.KvCache(ck, cv)

    return (lambda ck, cv, ks=None, vs=None, **a: api.paged_attention(cache=held(ck, cv, ks, vs), **a)), a


def plan_call(api, _):
    i = torch.int32
    return api.tree_plan, dict(parents=t(i, 7), q_start=t(i, 3), seq_lens=t(i, 2), masks=t(torch.int64, 7), positions=t(i, 7), ws=t(torch.uint8, 1024))


@pytest.mark.parametrize("make,codes,name", [(attention_call, False, "moe_paged_tree_attention"), (attention_call, True, "moe_paged_attention8"),
                                             (plan_call, False, "moe_tree_plan")])
def test_binding_refuses_tensors_elsewhere(api, calls, make, codes, name):
    fn, tensors = make(api, codes)
    fn(**tensors)
    assert calls.made == [name]
    for arg, x in tensors.items():
        plain = x.as_subclass(torch.Tensor)
        for wrong in (plain.as_subclass(OnHost), plain.as_subclass(OnOtherGpu), plain.double().as_subclass(OnGpu)):
            with pytest.raises(api.MoeError):
                fn(**{**tensors, arg: wrong})
    with pytest.raises(api.MoeError):
        fn(**tensors, **({"window": 3} if make is attention_call else {"stream": type("S", (), dict(device_index=1, cuda_stream=5))}))
    assert len(calls.made) == 1


@pytest.mark.parametrize("name,codes", NAMES)
def test_binding_lets_calls_without_tokens_through(api, calls, name, codes):
    fn, a = binding_call(api, name, codes)
    none = {n: x[:0] if n not in ("turns", "ws", "ck", "cv", "ks", "vs") else x for n, x in a.items()}
    fn(**none)
    assert len(calls.made) == 1
