"""Rotary positions, alone and in one pass with the write into a cache, and the
cache of 8-bit values (write and read back) against plain 64-bit references
(tests/cache8_util.py)."""
import math

import numpy as np
import pytest
import torch

from cache8_util import by_slot, dequantise, make_cache8, quantise, rotate
from paged_util import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_rotated(got, x, positions, r):
    """Half a step of the type; the angle's rounding to fp32 (2^-24 of at most
    pi/4), cos and sin (two steps each), the factor, the products and their sum:
    less than 8 * 2^-24 of |first| + |second|. Below the type's smallest normal
    value its step is absolute."""
    want, mag = rotate(x.double(), positions, r.turns, r.rotary_dim, r.interleaved, r.scale)
    t = torch.finfo(got.dtype)
    tol = t.eps / 2 * (want.abs() + 2.0 ** -21 * mag) + 2.0 ** -21 * mag + t.tiny * t.eps / 2
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() / tol).max())


@pytest.mark.parametrize("T,hq,hkv,d,rd,pairs,dtype,scaling,top", [
    (1, 1, 0, 64, 64, "half", torch.bfloat16, "none", 5),
    (3, 5, 1, 128, 128, "half", torch.bfloat16, "linear", 1 << 30),
    (7, 32, 8, 128, 64, "interleaved", torch.float16, "ntk", 5000),
    (33, 8, 2, 64, 16, "half", torch.float16, "yarn", 200000),
    (64, 7, 3, 192, 48, "half", torch.bfloat16, "bands", 200000),
    (5, 2, 2, 512, 512, "interleaved", torch.bfloat16, "yarn", (1 << 31) - 1),
    (9, 3, 1, 80, 80, "half", torch.float16, "none", 300),
    (4, 40, 1, 16, 16, "interleaved", torch.bfloat16, "none", 300),
    (2500, 12, 4, 128, 96, "half", torch.bfloat16, "none", 131072),
    (40, 3, 0, 160, 32, "interleaved", torch.float16, "none", 99),
])
@pytest.mark.parametrize("place", ["out", "in"])
def test_rope(api, T, hq, hkv, d, rd, pairs, dtype, scaling, top, place):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    fused = torch.empty((T, hq + hkv + 1, d), device="cuda").normal_(generator=g).to(dtype)
    q, k = fused[:, 1:1 + hq], fused[:, 1 + hq:] if hkv else None
    positions = torch.randint(0, top, (T,), device="cuda", generator=g).int()
    positions[0] = top - 1
    if T > 4:
        positions[T // 2] = -1
        positions[-1] = -5
    r = api.Rope(rd, base=10000.0 if T % 2 else 500000.0, interleaved=pairs == "interleaved", scaling=scaling,
                 factor=1.0 if scaling == "none" else 8.0, context=0 if scaling == "none" else 4096)
    was = fused.clone()
    if place == "in":
        api.rope(q, k, positions, r)
        new_q, new_k, keep_q, keep_k = q, k, was[:, 1:1 + hq], was[:, 1 + hq:]
        assert torch.equal(fused[:, 0], was[:, 0])
    else:
        # outputs of strides of their own: heads before tokens
        out = torch.full((hq + hkv, T, d + 16), 7.0, dtype=dtype, device="cuda")[..., :d].transpose(0, 1)
        new_q, new_k = out[:, :hq], out[:, hq:] if hkv else None
        keep_q, keep_k = new_q.clone(), new_k.clone() if hkv else None
        api.rope(q, k, positions, r, q_out=new_q, k_out=new_k)
        assert torch.equal(fused, was)
    assert api.last_launch_count() == 1
    real = positions >= 0
    pairs_of = [(new_q, was[:, 1:1 + hq], keep_q)] + ([(new_k, was[:, 1 + hq:], keep_k)] if hkv else [])
    for new, x, keep in pairs_of:
        assert torch.equal(new[~real], keep[~real])
        check_rotated(new[real], x[real], positions[real], r)
        assert torch.equal(new[real][..., rd:], x[real][..., rd:])


def test_rope_of_any_frequencies(api):
    """Half a turn, a quarter and none a position: exact whatever the position."""
    f = [math.pi, math.pi / 2, 0.0, -math.pi / 2] * 2
    r = api.Rope.of(f)
    assert r.turns.tolist() == [-(1 << 63), 1 << 62, 0, -(1 << 62)] * 2
    x = torch.randn((6, 2, 32), device="cuda").bfloat16()
    positions = i32([0, 1, 2, 3, (1 << 31) - 1, (1 << 31) - 2])
    y = torch.empty_like(x)
    api.rope(x, None, positions, r, q_out=y)
    for t, p in enumerate(positions.tolist()):
        a, b = x[t, :, :8].double(), x[t, :, 8:16].double()
        z = torch.complex(a, b) * torch.tensor([1j ** ((n * p) % 4) for n in (2, 1, 0, 3)] * 2, device="cuda")
        assert torch.equal(y[t, :, :8].double(), z.real) and torch.equal(y[t, :, 8:16].double(), z.imag)
    assert torch.equal(y[..., 16:], x[..., 16:])


def slots_of(T, room, seed):
    """T different slots with some of none among them."""
    s = torch.from_numpy(np.random.RandomState(seed).permutation(room)[:T].astype(np.int32)).cuda()
    if T > 3:
        s[T // 2] = -1
    return s


def inputs8(T, heads, d, dtype, seed):
    """Keys and values of sizes from the type's smallest to its largest, rows of
    zeros, borders of the scale and ties of the codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((2, T, heads, d), dtype=torch.float64, device="cuda").normal_(generator=g)
    top = 120 if dtype == torch.bfloat16 else 12
    low = -130 if dtype == torch.bfloat16 else -22
    x *= torch.exp2(torch.randint(low, top, (2, T, heads, 1), device="cuda", generator=g).double())
    x[0, 0] = 0.0
    if T > 2:
        x[1, 1, 0] = torch.arange(d, device="cuda") * 28.0 / 8          # 448 / 128 steps: codes and ties between them
        x[1, 1, 0, -1] = 448.0
        x[0, 2, 0] = torch.arange(d, device="cuda") / 8
        x[0, 2, 0, 0] = 450.0                                           # just above a border (449 where the type holds it)
        x[1, 2, -1, :] = 2.0 ** -8
        x[1, 2, -1, 3] = 1.0
    return x.to(dtype)


@pytest.mark.parametrize("T,heads,d,page,dtype,layout", [(1, 1, 64, 16, torch.bfloat16, "bthd"), (37, 5, 128, 16, torch.float16, "bhtd"),
                                                         (515, 8, 128, 48, torch.bfloat16, "pair"), (2000, 2, 64, 1024, torch.float16, "bthd"),
                                                         (300, 3, 128, 32, torch.bfloat16, "bthd")])
def test_append8_and_read8(api, T, heads, d, page, dtype, layout):
    n_blocks = T // page + 4
    cache = make_cache8(api, n_blocks, page, heads, d, layout)
    before = by_slot(cache)
    kv = inputs8(T, heads, d, dtype, T)
    fused = torch.zeros((T, 2 * heads + 1, d), dtype=dtype, device="cuda")
    fused[:, :heads], fused[:, heads + 1:] = kv[0], kv[1]
    slots = slots_of(T, n_blocks * page, T)
    ws = api.paged_workspace()
    api.paged_append(fused[:, :heads], fused[:, heads + 1:], slots, cache, ws)
    assert api.last_launch_count() == 1 and api.read_status(ws) == 0
    at = slots.cpu().numpy()
    live = at >= 0
    want = []
    for (codes, byte), (codes0, byte0), x in zip(by_slot(cache), before, kv):
        c, b = quantise(x.double().cpu().numpy())
        codes0[at[live]], byte0[at[live]] = c[live], b[live]
        assert (byte == byte0).all()
        # (a zero keeps its sign or not: the value is the same)
        assert (np.where(codes == 128, 0, codes) == np.where(codes0 == 128, 0, codes0)).all()
        want.append(dequantise(c, b))
    for out_type in (torch.bfloat16, torch.float16):
        out = torch.full((2, heads, T, d + 8), 3.0, dtype=out_type, device="cuda")[..., :d].transpose(1, 2)
        api.paged_read(cache, slots, out[0], out[1], ws)
        assert api.last_launch_count() == 1 and api.read_status(ws) == 0
        for o, w in zip(out, want):
            # one rounding of the value, as torch's from 64 bits (but for its way by fp32: e4m3 times a power of two fits that)
            w = torch.from_numpy(w).cuda().float().to(out_type)
            w[torch.from_numpy(~live).cuda()] = 3.0
            assert torch.equal(o, w)


def test_append8_again_gives_the_same_values(api):
    cache, again = make_cache8(api, 9, 16, 4, 128), make_cache8(api, 9, 16, 4, 128)
    x = inputs8(120, 4, 128, torch.bfloat16, 5)
    # (values that stay normal in bf16 on the way: bytes of at least 20)
    x = torch.where(x.double().abs().amax(-1, keepdim=True) < 2.0 ** -90, torch.zeros_like(x), x)
    slots = torch.randperm(144, device="cuda")[:120].int()
    ws = api.paged_workspace()
    out = torch.empty((2, 2, 120, 4, 128), dtype=torch.bfloat16, device="cuda")
    api.paged_append(x[0], x[1], slots, cache, ws)
    api.paged_read(cache, slots, out[0, 0], out[0, 1], ws)
    api.paged_append(out[0, 0], out[0, 1], slots, again, ws)
    api.paged_read(again, slots, out[1, 0], out[1, 1], ws)
    assert torch.equal(out[0], out[1]) and api.read_status(ws) == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append8_of_what_is_not_finite(api, bad):
    """That token's head is NaN whole; its neighbours are as they would be."""
    cache, ws = make_cache8(api, 2, 16, 3, 64), api.paged_workspace()
    x = torch.randn((2, 5, 3, 64), device="cuda").bfloat16()
    x[0, 2, 1, 63] = bad
    x[1, 4, 0, 0] = bad
    slots = i32([3, 17, 8, 9, 31])
    api.paged_append(x[0], x[1], slots, cache, ws)
    out = torch.empty_like(x)
    api.paged_read(cache, slots, out[0], out[1], ws)
    gone = torch.zeros((2, 5, 3), dtype=torch.bool, device="cuda")
    gone[0, 2, 1] = gone[1, 4, 0] = True
    assert out[gone].isnan().all() and torch.isfinite(out[~gone]).all()
    # half a step of 3 bits at the most
    err = (out[~gone].double() - x[~gone].double()).abs()
    assert (err <= 2.0 ** -4 * x[~gone].double().abs() + 2.0 ** -10 * x[~gone].double().abs().amax(-1, keepdim=True) / 224).all()


@pytest.mark.parametrize("codes", [False, True])
def test_bad_slots_are_reported_and_left_out(api, codes):
    cache = make_cache8(api, 3, 16, 2, 64) if codes else api.KvCache(*make_cache(3, 16, 2, 64, torch.bfloat16, 1))
    x = torch.randn((2, 4, 2, 64), device="cuda").bfloat16()
    slots, good = i32([5, 48, -2, 47]), i32([5, -1, -1, 47])
    r, positions = api.Rope(64), i32([0, 1, 2, 3])
    for call in ("append", "rope_append", "read"):
        ws = api.paged_workspace()
        out, out2 = (torch.full_like(x, 2.0) for _ in range(2))
        for s, o in ((slots, out), (good, out2)):
            if call == "append":
                api.paged_append(x[0], x[1], s, cache, ws)
            elif call == "rope_append":
                api.paged_rope_append(x[0], x[0], x[1], positions, s, r, cache, ws, q_out=o[0])
            else:
                api.paged_read(cache, s, o[0], o[1], ws)
            if s is slots:
                assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
        assert torch.equal(out, out2)


def test_read_of_16_bits(api):
    for dtype, layout, d in ((torch.bfloat16, "bthd", 128), (torch.float16, "bhtd", 64), (torch.bfloat16, "pair", 64)):
        k, v = make_cache(20, 24, 3, d, dtype, 4, layout)
        slots = torch.randint(0, 480, (777,), device="cuda").int()  # some more than once
        slots[5] = -1
        out = torch.full((2, 777, 3, d), 9.0, dtype=dtype, device="cuda")
        ws = api.paged_workspace()
        api.paged_read(api.KvCache(k, v), slots, out[0], out[1], ws)
        live = slots >= 0
        for o, c in zip(out, (k, v)):
            s = slots.long().clamp_min(0)
            assert torch.equal(o[live], c[s // 24, s % 24][live]) and (o[~live] == 9.0).all()
        assert api.read_status(ws) == 0


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rd,pairs,dtype", [(1, 4, 1, 64, 64, "half", torch.bfloat16), (50, 12, 3, 128, 64, "half", torch.float16),
                                                       (700, 8, 8, 128, 128, "interleaved", torch.bfloat16), (6, 0, 5, 64, 32, "half", torch.bfloat16),
                                                       (2000, 32, 8, 128, 128, "half", torch.bfloat16)])
def test_one_pass_is_the_two_calls(api, codes, T, hq, hkv, d, rd, pairs, dtype):
    page, n_blocks = 16, T // 16 + 3
    g = torch.Generator(device="cuda").manual_seed(T)
    fused = torch.empty((T, hq + 2 * hkv, d), device="cuda").normal_(generator=g).to(dtype)
    q, k, v = fused[:, :hq] if hq else None, fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    slots = slots_of(T, n_blocks * page, T)
    positions = torch.randint(0, 100000, (T,), device="cuda", generator=g).int()
    if T > 20:
        positions[T - 7:] = -1  # padding, whatever its slots say
    r = api.Rope(rd, interleaved=pairs == "interleaved", scale=1.25)

    def cache():
        if codes:
            return make_cache8(api, n_blocks, page, hkv, d)
        return api.KvCache(*(torch.full((n_blocks, page, hkv, d), 5.0, dtype=dtype, device="cuda") for _ in range(2)))

    one, two, ws = cache(), cache(), api.paged_workspace()
    was = fused.clone()
    q1 = torch.full((T, hq, d), 3.0, dtype=dtype, device="cuda") if hq else None
    api.paged_rope_append(q, k, v, positions, slots, r, one, ws, q_out=q1)
    assert api.last_launch_count() == 1 and torch.equal(fused, was)
    k2 = k.clone()
    q2 = torch.full((T, hq, d), 3.0, dtype=dtype, device="cuda") if hq else None
    if hq:
        api.rope(q, k2, positions, r, q_out=q2)
        assert torch.equal(q1, q2)
    else:
        api.rope(k2, None, positions, r)
    api.paged_append(k2, v, torch.where(positions >= 0, slots, -1), two, ws)
    assert torch.equal(one.k, two.k) and torch.equal(one.v, two.v)
    if codes:
        assert torch.equal(one.k_scale, two.k_scale) and torch.equal(one.v_scale, two.v_scale)
    assert api.read_status(ws) == 0
    if hq:  # and in place
        api.paged_rope_append(q, k, v, positions, slots, r, one, ws)
        assert torch.equal(q[positions >= 0], q2[positions >= 0]) and torch.equal(fused[:, hq:], was[:, hq:])
        assert torch.equal(q[positions < 0], was[:, :hq][positions < 0])


def test_captured_on_another_stream(api):
    """The write and the reading back as a graph, replayed on new tokens."""
    T, hq, hkv, d = 40, 8, 2, 128
    cache, ws, r = make_cache8(api, 8, 16, hkv, d), api.paged_workspace(), api.Rope(d)
    fused = torch.zeros((T, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    slots, positions = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    q, out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((2, T, hkv, d), dtype=torch.bfloat16, device="cuda")

    def step():
        api.paged_rope_append(fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:], positions, slots, r, cache, ws, q_out=q)
        api.paged_read(cache, slots, out[0], out[1], ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in (1, 2):
            torch.manual_seed(seed)
            fused.normal_()
            slots.copy_(torch.randperm(128, device="cuda")[:T])
            positions.copy_(torch.randint(0, 9999, (T,), device="cuda"))
            out.zero_()
            graph.replay()
            got = q.clone(), out.clone()
            q.zero_(), out.zero_()
            step()
            assert torch.equal(q, got[0]) and torch.equal(out, got[1])
    torch.cuda.current_stream().wait_stream(stream)
    assert api.read_status(ws) == 0
