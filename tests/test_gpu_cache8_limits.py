"""The cache of 8-bit values at the ends of its range, and one workspace for the
attentions over both kinds of cache."""
import math

import numpy as np
import pytest
import torch

import paged_util
from cache8_util import by_slot, check_attention8, dequantise, make_cache8, make_step8

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    a.set_option(a.OPT_GRID_CTAS, 0)
    return a


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def next_to_the_largest(dtype, d):
    """[8, 1, d]: the type's largest value, the tie of codes below it (248 times a
    power of two), what lies around them, and rows without any of that."""
    t = torch.finfo(dtype)
    by = t.max * (1 + t.eps / 2) / 256  # the largest value is just below 256 of these
    by = 2.0 ** round(math.log2(by))
    x = torch.randn((8, 1, d), dtype=torch.float64, generator=torch.Generator().manual_seed(3)) * by * 50
    x[0, 0, 0] = t.max
    x[1, 0, 1] = -t.max
    x[2, 0, 2] = 248 * by
    x[3, 0, 3], x[3, 0, 4] = 248 * by * (1 - t.eps), -240 * by  # one step below the tie
    x[4, 0, :] = t.max
    x[5, 0, 5], x[5, 0, 6] = 250 * by, -t.max
    x[6, 0, 0] = 240 * by
    return x.to(dtype).cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rotated", [False, True])
def test_values_next_to_the_largest_stay_finite(api, dtype, d, rotated):
    """Written, read back and written again, as an accepted path is: the same
    values, each within half a step of its code (2^-4 of it, or of the head's
    smallest normal code) of what was written."""
    x = next_to_the_largest(dtype, d)
    cache, again, ws = make_cache8(api, 1, 16, 1, d), make_cache8(api, 1, 16, 1, d), api.paged_workspace()
    slots = i32([3, 0, 15, 7, 8, 1, 4, 9])
    out = torch.zeros((2, 2, *x.shape), dtype=dtype, device="cuda")

    def write(k, v, c):
        if rotated:  # by no turn at all
            api.paged_rope_append(None, k, v, i32([0] * 8), slots, api.Rope(d), c, ws)
        else:
            api.paged_append(k, v, slots, c, ws)

    write(x, x.flip(2).contiguous(), cache)
    api.paged_read(cache, slots, out[0, 0], out[0, 1], ws)
    write(out[0, 0], out[0, 1], again)
    api.paged_read(again, slots, out[1, 0], out[1, 1], ws)
    assert api.read_status(ws) == 0
    assert torch.isfinite(out).all() and torch.equal(out[0], out[1])
    for a, b in zip(by_slot(cache), by_slot(again)):
        at = slots.cpu().numpy()
        assert np.array_equal(dequantise(a[0][at], a[1][at]), dequantise(b[0][at], b[1][at]))
    for o, want in ((out[0, 0], x), (out[0, 1], x.flip(2))):
        o, want = o.double(), want.double()
        assert ((o - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * want.abs().amax(-1, keepdim=True) / 224).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_over_the_largest_values_is_finite(api, dtype):
    """A row that sees one token has that token's values."""
    x = next_to_the_largest(dtype, 64)
    cache, ws = make_cache8(api, 8, 16, 1, 64), api.paged_workspace(1, make_cache8(api, 8, 16, 1, 64))
    slots = i32([16 * i for i in range(8)])
    api.paged_append(torch.zeros_like(x), x, slots, cache, ws)
    back, out = torch.empty((2, *x.shape), dtype=dtype, device="cuda"), torch.empty_like(x)
    api.paged_read(cache, slots, back[0], back[1], ws)
    q = torch.randn((8, 1, 64), device="cuda").to(dtype)
    api.paged_attention(q, cache, i32([[i] for i in range(8)]), i32(list(range(9))), i32([1] * 8), out, ws)
    assert api.read_status(ws) == 0 and torch.isfinite(out).all()
    want = back[1].double()
    # the weight is 2^11, by its reference's rounding (2^-20 for scores below 16) and that of four powers (2^-22 each) off from the sum's; then
    # the output's own
    assert ((out.double() - want).abs() <= (torch.finfo(dtype).eps / 2 + 2.0 ** -18) * want.abs()).all()


@pytest.mark.parametrize("d", [64, 128])
def test_queries_up_to_the_largest(api, d):
    """One large element of a query against a small one of a key: the scores are
    some 2^8, the row's factor alone passes fp32's range. Every third row of an
    item is of usual size."""
    e = torch.tensor([100, 120, 124, 125, 126, 126, 127, 127], device="cuda")  # by head
    s = make_step8(api, [(300, 20), (33, 2)], 16, 8, 8, d, torch.bfloat16, 7, spread=(0.5, 0.5))
    cache, g = s["cache"], torch.Generator(device="cuda").manual_seed(1)
    y = torch.empty(cache.k.shape, device="cuda").normal_(generator=g) * (64 / d) ** 0.5
    y[..., 0] = 2.0 ** -9
    y = y.to(torch.float8_e4m3fn)
    real = cache.k_scale != 255
    cache.k.copy_(y.view(torch.uint8))
    byte = (25 + 127 - e).to(torch.uint8)[None, :, None].expand_as(cache.k_scale)
    cache.k_scale.copy_(torch.where(real, byte, cache.k_scale))
    s["k"] = y.double() * torch.exp2((25 - e).double())[None, None, :, None]
    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda").normal_(generator=g) * 2.0 ** -20
    q[..., 0] = 1.0
    q *= torch.exp2(e.double())[None, :, None]
    q[1::3] *= 2.0 ** -60
    s["q"] = q.bfloat16()
    ws = api.paged_workspace(8, cache)
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    api.paged_attention(s["q"], cache, s["table"], s["q_start"], s["seq"], out, ws, lse=lse, scale=2.0 ** -8)
    assert api.read_status(ws) == 0
    ref = paged_util.attention(s, 2.0 ** -8)
    check_attention8(out, None, ref, 300)
    # a score of 2^8 is off by its rounding and its factor's, 2^-24 of it each, and by its products'
    assert ((lse.double() - ref[1]).abs() <= 2.0 ** -13 + 2.0 ** -20 * ref[1].abs()).all()


@pytest.mark.parametrize("dtype,by", [(torch.bfloat16, (119, 110, 60, -60, -112, -117)), (torch.float16, (13, 12, 0, -4, -9, -14))])
@pytest.mark.parametrize("d", [64, 128])
def test_values_up_to_the_largest(api, dtype, by, d):
    """Heads of values from the type's largest to its smallest, over many keys:
    sums of weights times values pass fp32's range where the outputs do not."""
    lens = [(3000, 20), (20000, 1), (5, 5)]
    s = make_step8(api, lens, 16, 12, 6, d, dtype, 6, spread=(0.3, 0.0))
    e = torch.tensor(by, device="cuda")
    real = s["cache"].v_scale != 255
    s["cache"].v_scale.copy_(torch.where(real, (s["cache"].v_scale.int() + e.int()[None, :, None]).to(torch.uint8), s["cache"].v_scale))
    s["v"] = s["v"] * torch.exp2(e.double())[None, None, :, None]
    ws = api.paged_workspace(12, s["cache"])
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    api.paged_attention(s["q"], s["cache"], s["table"], s["q_start"], s["seq"], out, ws, lse=lse)
    assert api.read_status(ws) == 0
    check_attention8(out, lse, paged_util.attention(s), 20000)


def test_one_workspace_for_both_attentions(api):
    """Calls over both kinds of cache in turn, of few and of many rows, on a buffer
    of the larger size, zeroed once: each as on a workspace of its own."""
    lens = [(3000, 300), (700, 6), (90, 90), (5000, 1), (64, 20)]
    a = paged_util.make_step(lens, 16, 32, 8, 128, torch.bfloat16, 31)
    b = make_step8(api, lens, 16, 32, 8, 128, torch.bfloat16, 32)
    small = make_step8(api, [(1500, 2), (40, 1)], 16, 8, 2, 64, torch.float16, 33)
    cache = api.KvCache(a["k"], a["v"])
    runs = [(a, cache), (b, b["cache"]), (small, small["cache"])]

    def call(s, c, ws):
        out = torch.full_like(s["q"], 3.0)
        api.paged_attention(s["q"], c, s["table"], s["q_start"], s["seq"], out, ws)
        assert api.read_status(ws) == 0
        return out

    want = [call(s, c, api.paged_workspace(s["q"].shape[1], c)) for s, c in runs]
    sizes = [api.paged_workspace(s["q"].shape[1], c).numel() for s, c in runs]
    assert max(sizes) == sizes[0]
    ws = api.paged_workspace(32, cache)
    for ctas in (0, 7, 152, 0):
        api.set_option(api.OPT_GRID_CTAS, ctas)
        try:
            got = [call(s, c, ws) for _ in range(2) for s, c in runs]
        finally:
            api.set_option(api.OPT_GRID_CTAS, 0)
        if ctas in (0, 152):
            for g, w in zip(got, want * 2):
                assert torch.equal(g, w)
        assert int(ws[api.PAGED_WORKSPACE_BYTES:api.PAGED_WORKSPACE_BYTES + 3 * 4 * 256].count_nonzero()) == 0
