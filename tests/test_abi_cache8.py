"""Host-side refusals of rotary positions, the cache of 8-bit values and
reading back: every case returns its code before any launch (this suite also
runs without a GPU)."""
import ctypes

import pytest
import torch

from test_abi_paged import F, Calls, OnGpu, OnHost, OnOtherGpu, cache


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


def cache8(api, **over):
    f = dict(k=F, v=F, k_scale=F, v_scale=F, n_blocks=64, block_size=16, kv_heads=2, head_dim=64, k_block_stride=2048,
             k_token_stride=128, k_head_stride=64, v_block_stride=2048, v_token_stride=128, v_head_stride=64)
    f.update(over)
    return api._KvCache8(**f)


def angles(api, **over):
    f = dict(turns=F, rotary_dim=64, interleaved=0, scale=1.0)
    f.update(over)
    return api._RopeAngles(**f)


def call(api, name, c=None, a=None, **over):
    """The entry point `name` with arguments that it would take."""
    v = dict(q=F, qt=512, qh=64, qo=F + 65536, qot=512, qoh=64, hq=8, k=F, kt=128, kh=64, ko=F + 131072, kot=128, koh=64, hkv=2, v=F, vt=128,
             vh=64, T=4, d=64, dtype=0, positions=F, slots=F, ws=F, ws_bytes=1024)
    v.update(over)
    g = lambda names: [v[n] for n in names.split()]  # noqa: E731
    a = ctypes.byref(a or angles(api))
    c8, c16 = ctypes.byref(c or cache8(api)), ctypes.byref(c or cache(api))
    lib, q, kv, ws = api.lib, g("q qt qh qo qot qoh hq"), g("k kt kh v vt vh T"), g("ws ws_bytes") + [None]
    if name == "moe_rope":
        return lib.moe_rope(*q, *g("k kt kh ko kot koh hkv T d dtype positions"), a, None)
    if name == "moe_paged_rope_append":
        return lib.moe_paged_rope_append(*q, *kv, *g("positions slots"), a, c16, *ws)
    if name == "moe_paged_rope_append8":
        return lib.moe_paged_rope_append8(*q, *kv, *g("dtype positions slots"), a, c8, *ws)
    if name == "moe_paged_append8":
        return lib.moe_paged_append8(*kv, *g("dtype slots"), c8, *ws)
    if name == "moe_paged_read":
        return lib.moe_paged_read(c16, *g("slots T ko kot koh v vt vh"), *ws)
    return lib.moe_paged_read8(c8, *g("slots T dtype ko kot koh v vt vh"), *ws)


WITH_Q = ["moe_rope", "moe_paged_rope_append", "moe_paged_rope_append8"]
INTO_8 = ["moe_paged_rope_append8", "moe_paged_append8", "moe_paged_read8"]
READS = ["moe_paged_read", "moe_paged_read8"]
APPENDS = ["moe_paged_rope_append", "moe_paged_rope_append8", "moe_paged_append8"]


@pytest.mark.parametrize("name", INTO_8)
@pytest.mark.parametrize("over,code", [
    (dict(k=None), "EINVAL"), (dict(v_scale=None), "EINVAL"), (dict(head_dim=96), "ESHAPE"), (dict(kv_heads=0), "ESHAPE"),
    (dict(kv_heads=300), "ESHAPE"), (dict(block_size=8), "ESHAPE"), (dict(block_size=24), "ESHAPE"), (dict(block_size=2048), "ESHAPE"),
    (dict(n_blocks=0), "ESHAPE"), (dict(n_blocks=1 << 27), "ESHAPE"), (dict(k_token_stride=136), "ESHAPE"), (dict(v_head_stride=48), "ESHAPE"),
    (dict(v_block_stride=-2048), "ESHAPE"), (dict(k=F + 8), "EALIGN"), (dict(k_scale=F + 8), "EALIGN")], ids=lambda v: str(v))
def test_caches8(api, name, over, code):
    assert call(api, name, c=cache8(api, **over)) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("name", ["moe_paged_rope_append", "moe_paged_read"])
@pytest.mark.parametrize("over,code", [(dict(k=None), "EINVAL"), (dict(dtype=2), "ESHAPE"), (dict(block_size=20), "ESHAPE"), (dict(v=F + 2), "EALIGN")],
                         ids=lambda v: str(v))
def test_caches(api, name, over, code):
    assert call(api, name, c=cache(api, **over)) == getattr(api, code)


@pytest.mark.parametrize("name", WITH_Q)
@pytest.mark.parametrize("over,code", [
    (dict(turns=None), "EINVAL"), (dict(rotary_dim=8), "ESHAPE"), (dict(rotary_dim=40), "ESHAPE"), (dict(rotary_dim=80), "ESHAPE"),
    (dict(interleaved=2), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(turns=F + 4), "EALIGN")],
    ids=lambda v: str(v))
def test_angles(api, name, over, code):
    assert call(api, name, a=angles(api, **over)) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("name", WITH_Q)
@pytest.mark.parametrize("over,code", [
    (dict(T=-1), "ESHAPE"), (dict(hq=1025), "ESHAPE"), (dict(hq=-1), "ESHAPE"), (dict(qt=516), "ESHAPE"), (dict(qh=-64), "ESHAPE"),
    (dict(qot=32), "ESHAPE"), (dict(qoh=8), "ESHAPE"), (dict(q=F + 8), "EALIGN"), (dict(qo=F + 2), "EALIGN"), (dict(qo=None), "EINVAL"),
    (dict(qo=F, qot=1024), "EINVAL"), (dict(positions=None), "EINVAL"), (dict(positions=F + 2), "EALIGN"), (dict(kt=4), "ESHAPE")],
    ids=lambda v: str(v))
def test_rotations(api, name, over, code):
    assert call(api, name, **over) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("over,code", [
    (dict(d=24), "ESHAPE"), (dict(d=528), "ESHAPE"), (dict(dtype=2), "ESHAPE"), (dict(hq=0), "ESHAPE"), (dict(hkv=0), "ESHAPE"),
    (dict(k=None), "ESHAPE"), (dict(hkv=1025), "ESHAPE"), (dict(q=None), "EINVAL"), (dict(ko=None), "EINVAL"), (dict(koh=0), "ESHAPE"),
    (dict(k=F + 2), "EALIGN"), (dict(ko=F, koh=128), "EINVAL")], ids=lambda v: str(v))
def test_rope(api, over, code):
    assert call(api, "moe_rope", **over) == getattr(api, code)


@pytest.mark.parametrize("name", APPENDS)
@pytest.mark.parametrize("over,code", [
    (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(slots=None), "EINVAL"), (dict(T=-3), "ESHAPE"), (dict(vt=2), "ESHAPE"),
    (dict(vh=-8), "ESHAPE"), (dict(k=F + 4), "EALIGN"), (dict(v=F + 8), "EALIGN"), (dict(slots=F + 1), "EALIGN"), (dict(ws=None), "EWORKSPACE"),
    (dict(ws=F + 8), "EALIGN"), (dict(ws_bytes=1023), "EWORKSPACE")], ids=lambda v: str(v))
def test_appends(api, name, over, code):
    assert call(api, name, **over) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("name", ["moe_paged_rope_append8", "moe_paged_append8", "moe_paged_read8"])
def test_types(api, name):
    assert call(api, name, dtype=2) == call(api, name, dtype=-1) == api.ESHAPE


def test_queries_without_heads_or_heads_without_queries(api):
    for name in WITH_Q[1:]:
        assert call(api, name, q=None) == call(api, name, hq=0) == api.ESHAPE


@pytest.mark.parametrize("name", READS)
@pytest.mark.parametrize("over,code", [
    (dict(ko=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(slots=None), "EINVAL"), (dict(T=-1), "ESHAPE"), (dict(kot=32), "ESHAPE"),
    (dict(vh=0), "ESHAPE"), (dict(koh=68), "ESHAPE"), (dict(ko=F + 8), "EALIGN"), (dict(slots=F + 2), "EALIGN"), (dict(ws=None), "EWORKSPACE"),
    (dict(ws=F + 4), "EALIGN"), (dict(ws_bytes=8), "EWORKSPACE")], ids=lambda v: str(v))
def test_reads(api, name, over, code):
    assert call(api, name, **over) == getattr(api, code)
    assert api.last_launch_count() == 0


@pytest.mark.parametrize("name", WITH_Q + APPENDS[2:] + READS)
def test_nothing_to_do(api, name):
    assert call(api, name, T=0, slots=None, positions=None, v=None, ko=None, ws=None) == api.OK
    assert api.last_launch_count() == 0


# ------------------------------------------------------------------ the binding
def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def rope_of(api, turns):
    r = api.Rope(64, device="cpu")
    r.turns, r.device_index = turns, turns.get_device()
    return r


def binding_call(api, name, codes):
    i, b, u8 = torch.int32, torch.bfloat16, torch.uint8
    kv = dict(ck=t(u8 if codes else b, 8, 16, 2, 64), cv=t(u8 if codes else b, 8, 16, 2, 64))
    if codes:
        kv.update(ks=t(u8, 8, 2, 16), vs=t(u8, 8, 2, 16))

    def held(ck, cv, ks=None, vs=None):
        return api.KvCache8(ck, cv, ks, vs) if codes else api.KvCache(ck, cv)

    turns, ws = t(torch.int64, 32), t(u8, 1024)
    if name == "rope":
        a = dict(q=t(b, 3, 4, 64), k=t(b, 3, 2, 64), positions=t(i, 3), q_out=t(b, 3, 4, 64), k_out=t(b, 3, 2, 64), turns=turns)
        return (lambda turns, **a: api.rope(angles=rope_of(api, turns), **a)), a
    new = dict(k_new=t(b, 3, 2, 64), v_new=t(b, 3, 2, 64), slot_map=t(i, 3), ws=ws, **kv)
    if name == "paged_append":
        return (lambda ck, cv, ks=None, vs=None, **a: api.paged_append(cache=held(ck, cv, ks, vs), **a)), new
    if name == "paged_rope_append":
        a = dict(q=t(b, 3, 4, 64), positions=t(i, 3), q_out=t(b, 3, 4, 64), turns=turns, **new)
        return (lambda ck, cv, turns, ks=None, vs=None, **a: api.paged_rope_append(angles=rope_of(api, turns), cache=held(ck, cv, ks, vs), **a)), a
    a = dict(slot_map=t(i, 3), k_out=t(b, 3, 2, 64), v_out=t(b, 3, 2, 64), ws=ws, **kv)
    return (lambda ck, cv, ks=None, vs=None, **a: api.paged_read(cache=held(ck, cv, ks, vs), **a)), a


NAMES = [("rope", False), ("paged_append", True), ("paged_rope_append", False), ("paged_rope_append", True), ("paged_read", False), ("paged_read", True)]


@pytest.fixture
def calls(api, monkeypatch):
    calls = Calls(api.lib)
    calls.moe_rope_table = api.lib.moe_rope_table  # host code
    monkeypatch.setattr(api, "lib", calls)
    monkeypatch.setattr(api, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    return calls


@pytest.mark.parametrize("name,codes", NAMES)
def test_binding_refuses_tensors_elsewhere(api, calls, name, codes):
    """Each tensor of a call in turn in host memory, on another device, of
    another type: no address of it reaches the library."""
    fn, tensors = binding_call(api, name, codes)
    fn(**tensors)
    assert calls.made == ["moe_" + name + ("8" if codes else "")]
    for arg, x in tensors.items():
        for elsewhere in (OnHost, OnOtherGpu):
            with pytest.raises(api.MoeError):
                fn(**{**tensors, arg: x.as_subclass(torch.Tensor).as_subclass(elsewhere)})
        if arg != "turns":
            with pytest.raises(api.MoeError):
                fn(**{**tensors, arg: x.as_subclass(torch.Tensor).double().as_subclass(OnGpu)})

    class Stream:
        device_index, cuda_stream = 1, 5

    with pytest.raises(api.MoeError):
        fn(**tensors, stream=Stream)
    assert len(calls.made) == 1


@pytest.mark.parametrize("name,codes", NAMES)
def test_binding_refuses_other_shapes(api, calls, name, codes):
    fn, tensors = binding_call(api, name, codes)
    for arg, x in tensors.items():
        if arg in ("turns", "ws"):
            continue
        more = torch.zeros((x.shape[0] + 1, *x.shape[1:]), dtype=x.dtype).as_subclass(OnGpu)
        with pytest.raises(api.MoeError):
            fn(**{**tensors, arg: more})
    assert not calls.made


def test_binding_takes_any_stride_of_a_dimension_of_one(api, calls):
    base = torch.zeros(8192, dtype=torch.bfloat16)
    one = base.as_strided((1, 1, 64), (389, 7, 1)).as_subclass(OnGpu)
    api.rope(one, one, t(torch.int32, 1), rope_of(api, t(torch.int64, 32)))  # in place: the output's own strides
    a = calls.args[-1]
    assert a[1:3] == a[4:6] == (64, 64) and a[8:10] == a[11:13] == (64, 64)
    c = api.KvCache8(*(torch.zeros(8192, dtype=torch.uint8).as_strided((1, 16, 1, 64), (5, 64, 3, 1)).as_subclass(OnGpu) for _ in range(2)),
                     t(torch.uint8, 1, 1, 16), t(torch.uint8, 1, 1, 16))
    assert (c._c.k_block_stride, c._c.k_token_stride, c._c.k_head_stride) == (64, 64, 64)
    api.paged_rope_append(one, one, one, t(torch.int32, 1), t(torch.int32, 1), rope_of(api, t(torch.int64, 32)), c, t(torch.uint8, 1024))
    a = calls.args[-1]
    assert a[1:3] == a[4:6] == (64, 64) and a[8:10] == a[11:13] == (0, 0)


def test_binding_without_keys_or_queries(api, calls):
    q, p = t(torch.bfloat16, 3, 4, 64), t(torch.int32, 3)
    r = rope_of(api, t(torch.int64, 32))
    api.rope(q, None, p, r)
    assert calls.args[-1][7:14] == (None, 0, 0, None, 0, 0, 0)
    with pytest.raises(api.MoeError):
        api.rope(q, None, p, r, k_out=q)
    fn, a = binding_call(api, "paged_rope_append", True)
    fn(**{**a, "q": None, "q_out": None})
    assert calls.args[-1][:7] == (None, 0, 0, None, 0, 0, 0)
    with pytest.raises(api.MoeError):
        fn(**{**a, "q": None})
