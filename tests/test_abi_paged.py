"""Host-side refusals of the paged step's entry points: every case returns
its code before any launch (this suite also runs without a GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


F = 4096  # an aligned address that no refused call touches


def cache(api, **over):
    f = dict(k=F, v=F, dtype=0, n_blocks=64, block_size=16, kv_heads=2, head_dim=64, k_block_stride=2048,
             k_token_stride=128, k_head_stride=64, v_block_stride=2048, v_token_stride=128, v_head_stride=64)
    f.update(over)
    return api._KvCache(**f)


BAD_CACHES = [(dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(dtype=2), "ESHAPE"), (dict(head_dim=96), "ESHAPE"),
              (dict(kv_heads=0), "ESHAPE"), (dict(kv_heads=300), "ESHAPE"), (dict(block_size=4), "ESHAPE"),
              (dict(block_size=20), "ESHAPE"), (dict(block_size=2048), "ESHAPE"), (dict(n_blocks=0), "ESHAPE"),
              (dict(n_blocks=1 << 28), "ESHAPE"), (dict(k_token_stride=132), "ESHAPE"), (dict(v_head_stride=32), "ESHAPE"),
              (dict(k_block_stride=-2048), "ESHAPE"), (dict(k=F + 8), "EALIGN"), (dict(v=F + 2), "EALIGN")]


def attend(api, c=None, **over):
    a = dict(q=F, qt=512, qh=64, T=4, heads=8, tables=F, width=8, q_start=F, seq=F, B=2, scale=0.0, window=0, out=F,
             lse=F, ws=F, ws_bytes=1 << 30)
    a.update(over)
    return api.lib.moe_paged_attention(a["q"], a["qt"], a["qh"], a["T"], a["heads"], ctypes.byref(c or cache(api)), a["tables"],
                                       a["width"], a["q_start"], a["seq"], a["B"], a["scale"], a["window"], a["out"], a["lse"],
                                       a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,code", BAD_CACHES, ids=lambda v: str(v))
def test_caches(api, over, code):
    c = cache(api, **over)
    want = getattr(api, code)
    assert attend(api, c) == want
    assert api.lib.moe_paged_append(F, 128, 64, F, 128, 64, 4, F, ctypes.byref(c), F, 1024, None) == want
    assert api.lib.moe_paged_attention_workspace_bytes(8, ctypes.byref(c)) == 0
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("over,code", [
    (dict(heads=7), "ESHAPE"), (dict(heads=0), "ESHAPE"), (dict(heads=128), "ESHAPE"), (dict(T=-1), "ESHAPE"),
    (dict(T=1 << 30), "ESHAPE"), (dict(B=0), "ESHAPE"), (dict(B=4097), "ESHAPE"), (dict(width=0), "ESHAPE"),
    (dict(window=-1), "ESHAPE"), (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(q=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(tables=None), "EINVAL"), (dict(q_start=None), "EINVAL"),
    (dict(seq=None), "EINVAL"), (dict(q=F + 8), "EALIGN"), (dict(out=F + 4), "EALIGN"), (dict(lse=F + 2), "EALIGN"),
    (dict(tables=F + 1), "EALIGN"), (dict(qt=516), "ESHAPE"), (dict(qh=-64), "ESHAPE"), (dict(ws=None), "EWORKSPACE"),
    (dict(ws=F + 4), "EALIGN"), (dict(ws_bytes=1024), "EWORKSPACE")], ids=lambda v: str(v))
def test_attention(api, over, code):
    assert attend(api, **over) == getattr(api, code)
    assert api.last_launch_count() == 0


def test_nothing_to_do(api):
    assert attend(api, T=0, q=None, out=None) == api.OK
    c = cache(api)
    assert api.lib.moe_paged_append(None, 128, 64, None, 128, 64, 0, None, ctypes.byref(c), F, 1024, None) == api.OK


@pytest.mark.parametrize("at,value,code", [
    (0, None, "EINVAL"), (1, None, "EINVAL"), (2, 0, "ESHAPE"), (2, 4097, "ESHAPE"), (3, None, "EINVAL"), (4, -1, "ESHAPE"),
    (6, None, "EINVAL"), (7, 0, "ESHAPE"), (8, 0, "ESHAPE"), (9, None, "EINVAL"), (10, None, "EINVAL"), (11, None, "EINVAL"),
    (13, -2, "ESHAPE"), (14, None, "EINVAL"), (15, None, "EWORKSPACE"), (16, 512, "EWORKSPACE"), (9, F, "EINVAL"),
    (10, F, "EINVAL"), (14, F + 4 * 64, "EINVAL"), (0, F + 2, "EALIGN"), (12, F + 1, "EALIGN"), (15, F + 4, "EALIGN")])
def test_plan(api, at, value, code):
    args = [F, F, 2, F, 8, F + 4 * 64, F + 4096, 4, 16, F + 8192, F + 12288, F + 16384, F + 20480, 8, F + 24576, F, 1024, None]
    args[at] = value
    assert api.lib.moe_paged_plan(*args) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("at,value,code", [
    (0, None, "EINVAL"), (1, 2, "ESHAPE"), (2, 0, "ESHAPE"), (3, 0, "ESHAPE"), (3, 720897, "ESHAPE"), (4, 99, "ESHAPE"),
    (5, None, "EINVAL"), (10, None, "EINVAL"), (0, F + 2, "EALIGN"), (5, F + 2, "EALIGN"), (7, F + 1, "EALIGN")])
def test_sample(api, at, value, code):
    args = [F, 0, 4, 100, 100, F, F, F, F, F, F, F, None]
    args[at] = value
    assert api.lib.moe_sample(*args) == getattr(api, code)
    assert api.last_launch_count() == 0


def test_binding_refuses_wrong_tensors(api):
    f, b = torch.float32, torch.bfloat16
    with pytest.raises(api.MoeError):
        api.KvCache(torch.zeros((2, 16, 2, 64)), torch.zeros((2, 16, 2, 64)))           # fp32
    with pytest.raises(api.MoeError):
        api.KvCache(torch.zeros((2, 16, 2, 64), dtype=b), torch.zeros((2, 16, 1, 64), dtype=b))
    with pytest.raises(api.MoeError):
        api.sample(torch.zeros((2, 10), dtype=torch.float64), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    c = api.KvCache(torch.zeros((2, 16, 2, 64), dtype=b), torch.zeros((2, 16, 2, 64), dtype=b))
    with pytest.raises(api.MoeError):
        api.paged_append(torch.zeros((3, 2, 64), dtype=f), torch.zeros((3, 2, 64), dtype=f), torch.zeros(3, dtype=torch.int32), c,
                         torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(api.MoeError):
        api.paged_workspace(3, c)                                                       # 3 heads over 2
    n = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(api.MoeError):
        api.paged_plan(n, n, n, n.view(1, 2), 16, n, n, n, n, n)
