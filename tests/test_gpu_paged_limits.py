"""Calls of the 8-bit cache, of trees and of rotation at the largest sizes that
their contracts allow, and what captured steps share."""
import math

import pytest
import torch

import paged_util
from cache8_util import check_attention8, make_cache8, make_step8, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    a.set_option(a.OPT_GRID_CTAS, 0)
    return a


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attend(api, s, q=None, **kw):
    q = s["q"] if q is None else q
    ws = api.paged_workspace(q.shape[1], s["cache"])
    out, lse = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda"), torch.full(q.shape[:2], 3.0, device="cuda")
    api.paged_attention(q, s["cache"], s["table"], s["q_start"], s["seq"], out, ws, lse=lse, window=s["window"], **kw)
    assert api.read_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
def test_attention8_of_slices_of_a_projection(api, d):
    s = make_step8(api, [(700, 40), (90, 3)], 32, 12, 3, d, torch.bfloat16, 1)
    fused = torch.full((43, 18, d), math.nan, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:14] = s["q"]
    out, lse = attend(api, s, fused[:, 2:14])
    want = attend(api, s)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    by_head = s["q"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(attend(api, s, by_head)[0], want[0])


def test_attention8_of_4096_requests(api):
    lens = [(1 + (37 * i) % 50, 1 if i % 3 else 0) for i in range(4096)]
    s = make_step8(api, lens, 16, 2, 1, 64, torch.float16, 2)
    out, lse = attend(api, s)
    check_attention8(out, lse, paged_util.attention(s), 50)


def test_attention8_of_256_kv_heads(api):
    s = make_step8(api, [(33, 2), (300, 1)], 16, 512, 256, 64, torch.bfloat16, 3)
    out, lse = attend(api, s)
    check_attention8(out, lse, paged_util.attention(s), 300)


@pytest.mark.parametrize("tree", [False, True])
def test_attention8_up_to_the_last_position(api, tree):
    """Keys at the end of the positions that fit 32 bits, by a window; under a tree
    the context is the pages that the table names over and over."""
    page, d, last = 1024, 64, (1 << 31) - 1
    width = -(-last // page)
    cache, ws = make_cache8(api, 3, page, 1, d), api.paged_workspace(4, make_cache8(api, 3, page, 1, d))
    x = torch.randn((2, 3 * page, 1, d), device="cuda").bfloat16()
    api.paged_append(x[0], x[1], torch.arange(3 * page, device="cuda").int(), cache, ws)
    back = torch.empty_like(x)
    api.paged_read(cache, torch.arange(3 * page, device="cuda").int(), back[0], back[1], ws)
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -1], table[0, -2] = 2, 0
    n, window = 3, 200
    q, out = torch.randn((n, 4, d), device="cuda").bfloat16(), torch.empty((n, 4, d), dtype=torch.bfloat16, device="cuda")
    if tree:  # the end of a shorter context, of which all is seen
        seq, window = 2 * page, 0
        table, masks = i32([[0, 2]]), torch.tensor([1, 3, 5], dtype=torch.int64, device="cuda")
        api.paged_attention(q, cache, table, i32([0, n]), i32([seq]), out, ws, tree_masks=masks)
        seen = [list(range(seq - n)) + [seq - n + j for j in range(n) if int(masks[i]) >> j & 1] for i in range(n)]
        where = lambda j: (0 if j < page else 2) * page + j % page  # noqa: E731
    else:
        seq = last
        api.paged_attention(q, cache, table, i32([0, n]), i32([seq]), out, ws, window=window)
        seen = [list(range(seq - n + i - window + 1, seq - n + i + 1)) for i in range(n)]
        where = lambda j: (2 if j // page == width - 1 else 0) * page + j % page  # noqa: E731
    assert api.read_status(ws) == 0
    for i in range(n):
        at = torch.tensor([where(j) for j in seen[i]], device="cuda")
        k, v = (back[m][at, 0].double() for m in range(2))
        p = torch.softmax(q[i].double() @ k.T / 8, -1)
        tol = (2.0 ** -11 + 2.0 ** -14) * (p @ v.abs()) + 2.0 ** -9 * (p @ v).abs() + len(at) * 2.0 ** -27 / 224 * (p @ v.abs()).amax(-1, keepdim=True)
        assert ((out[i].double() - p @ v).abs() <= tol).all()


def test_rotation_of_1024_heads(api):
    x = torch.randn((3, 1024, 64), device="cuda").half()
    k = torch.randn((3, 1024, 64), device="cuda").half()
    r, positions = api.Rope(64), i32([0, 77, 1 << 30])
    out, k_out = torch.empty_like(x), torch.empty_like(k)
    api.rope(x, k, positions, r, q_out=out, k_out=k_out)
    for a, b in ((x, out), (k, k_out)):  # as 32 heads at a time
        for h in range(0, 1024, 256):
            want = torch.empty((3, 256, 64), dtype=torch.float16, device="cuda")
            api.rope(a[:, h:h + 256], None, positions, r, q_out=want)
            assert torch.equal(b[:, h:h + 256], want)


def test_two_captured_graphs_on_one_workspace(api):
    """Two steps of other requests over other caches, replayed in turn."""
    a = make_step8(api, [(3000, 2), (200, 20)], 16, 8, 2, 128, torch.bfloat16, 4)
    b = paged_util.make_step([(2000, 90), (700, 1)], 16, 8, 2, 128, torch.bfloat16, 5)
    kv = api.KvCache(b["k"], b["v"])
    ws = api.paged_workspace(8, kv)
    steps = [(a, a["cache"]), (b, kv)]
    outs = [torch.zeros_like(s["q"]) for s, _ in steps]

    def call(i):
        s, cache = steps[i]
        api.paged_attention(s["q"], cache, s["table"], s["q_start"], s["seq"], outs[i], ws)

    want = []
    for i in range(2):
        call(i)
        want.append(outs[i].clone())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in steps]
    with torch.cuda.stream(stream):
        for i, g in enumerate(graphs):
            with torch.cuda.graph(g, stream=stream):
                call(i)
        for o in outs:
            o.zero_()
        for i in (0, 1, 1, 0, 0, 1):
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(outs[i], want[i])
    torch.cuda.current_stream().wait_stream(stream)
    assert api.read_status(ws) == 0


def test_a_slot_read_many_times(api):
    cache, ws = make_cache8(api, 2, 16, 2, 64), api.paged_workspace()
    x = torch.randn((2, 32, 2, 64), device="cuda").bfloat16()
    api.paged_append(x[0], x[1], torch.arange(32, device="cuda").int(), cache, ws)
    slots = i32([5] * 40 + [31, 5, -1, 0])
    out = torch.full((2, 44, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    api.paged_read(cache, slots, out[0], out[1], ws)
    codes, byte = quantise(x.double().cpu().numpy())
    assert torch.equal(out[:, :40], out[:, :1].expand(-1, 40, -1, -1)) and torch.equal(out[:, 41], out[:, 0]) and (out[:, 42] == 3).all()
    assert torch.equal(cache.k_scale.transpose(1, 2).reshape(32, 2).cpu(), torch.from_numpy(byte[0]))
