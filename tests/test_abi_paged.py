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


class OnGpu(torch.Tensor):
    """A host tensor that passes for one on a GPU, where no call is made."""
    index = 0
    is_cuda = property(lambda self: self.index >= 0)

    def get_device(self):
        return self.index


class OnOtherGpu(OnGpu):
    index = 1


class OnHost(OnGpu):
    index = -1


class Calls:
    """Stands for the library: counts the calls that the binding lets through."""

    def __init__(self, lib):
        self.made, self.args, self.moe_status_str = [], [], lib.moe_status_str

    def __getattr__(self, name):
        return lambda *args: self.made.append(name) or self.args.append(args) or 0


def binding_call(api, name):
    """(function, its tensors by argument) of an accepted call."""
    def t(dtype, *shape):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)

    i, f, b = torch.int32, torch.float32, torch.bfloat16
    kv = dict(k=t(b, 8, 16, 2, 64), v=t(b, 8, 16, 2, 64))
    ws = t(torch.uint8, 1024)
    if name == "paged_plan":
        a = dict(ctx_lens=t(i, 2), new_lens=t(i, 2), free_list=t(i, 9), block_tables=t(i, 2, 4), q_start=t(i, 3), seq_lens=t(i, 2),
                 slot_map=t(i, 7), taken=t(i, 1), ws=ws, positions=t(i, 7), free_head=t(i, 1))
        return (lambda **a: api.paged_plan(block_size=16, **a)), a
    if name == "paged_append":
        a = dict(k_new=t(b, 3, 2, 64), v_new=t(b, 3, 2, 64), slot_map=t(i, 3), ws=ws, **kv)
        return (lambda k, v, **a: api.paged_append(cache=api.KvCache(k, v), **a)), a
    if name == "paged_attention":
        a = dict(q=t(b, 3, 4, 64), block_tables=t(i, 2, 4), q_start=t(i, 3), seq_lens=t(i, 2), out=t(b, 3, 4, 64), ws=ws,
                 lse=t(f, 3, 4), **kv)
        return (lambda k, v, **a: api.paged_attention(cache=api.KvCache(k, v), **a)), a
    a = dict(logits=t(f, 2, 10), u=t(f, 2), tokens=t(i, 2), probs=t(f, 2), temperature=t(f, 2), top_k=t(i, 2), top_p=t(f, 2),
             min_p=t(f, 2))
    return api.sample, a


@pytest.mark.parametrize("name", ["paged_plan", "paged_append", "paged_attention", "sample"])
def test_binding_refuses_tensors_elsewhere(api, monkeypatch, name):
    """Each tensor of a call in turn in host memory and on another device than
    the current one: no address of it reaches the library."""
    calls = Calls(api.lib)
    monkeypatch.setattr(api, "lib", calls)
    monkeypatch.setattr(api, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    call, tensors = binding_call(api, name)
    call(**tensors)
    assert calls.made == ["moe_" + name]
    for arg, t in tensors.items():
        for elsewhere in (OnHost, OnOtherGpu):
            with pytest.raises(api.MoeError):
                call(**{**tensors, arg: t.as_subclass(torch.Tensor).as_subclass(elsewhere)})
        if arg == "ws":
            for wrong in (torch.zeros(1024, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)[::4]):
                with pytest.raises(api.MoeError):
                    call(**{**tensors, arg: wrong.as_subclass(OnGpu)})

    if "k" in tensors:  # both of the cache's tensors
        for elsewhere in (OnHost, OnOtherGpu):
            with pytest.raises(api.MoeError):
                call(**{**tensors, **{n: tensors[n].as_subclass(torch.Tensor).as_subclass(elsewhere) for n in "kv"}})

    class Stream:
        device_index, cuda_stream = 1, 5

    with pytest.raises(api.MoeError):
        call(**tensors, stream=Stream)
    Stream.device_index = 0
    assert len(calls.made) == 1
    call(**tensors, stream=Stream)
    assert len(calls.made) == 2


def test_hold_back_is_off_or_on(api):
    for value, code in ((-1, api.EINVAL), (2, api.EINVAL), (0, api.OK)):
        assert api.lib.moe_set_option(api.OPT_DEBUG_HOLD_BACK, value) == code


def test_binding_takes_any_stride_of_a_dimension_of_one(api, monkeypatch):
    """One token, one head, one block: what a view says of the step along them
    (here not a multiple of 8) is not one that anything takes."""
    calls = Calls(api.lib)
    monkeypatch.setattr(api, "lib", calls)
    monkeypatch.setattr(api, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    base = torch.zeros(8192, dtype=torch.bfloat16)

    def view(shape, strides):
        return base.as_strided(shape, strides).as_subclass(OnGpu)

    for shape, strides in (((1, 16, 2, 64), (5, 128, 64, 1)), ((2, 16, 1, 64), (1024, 64, 3, 1)), ((1, 8, 1, 64), (0, 64, 7, 1))):
        cache = api.KvCache(view(shape, strides), view(shape, strides))
        assert all(getattr(cache._c, f"{n}_{w}_stride") % 8 == 0 and getattr(cache._c, f"{n}_{w}_stride") >= 64
                   for n in "kv" for w in ("block", "token", "head"))
    _, a = binding_call(api, "paged_append")
    api.paged_append(view((1, 1, 64), (389, 7, 1)), view((1, 1, 64), (3, 9, 1)), a["slot_map"][:1], cache, a["ws"])
    assert calls.args[-1][1:3] == calls.args[-1][4:6] == (0, 0)
    _, a = binding_call(api, "paged_attention")
    api.paged_attention(view((1, 1, 64), (389, 7, 1)), cache, a["block_tables"], a["q_start"], a["seq_lens"], view((1, 1, 64), (64, 64, 1)),
                        a["ws"])
    assert calls.args[-1][1:3] == (0, 0)
