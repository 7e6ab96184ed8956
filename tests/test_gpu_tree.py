"""Trees of drafted tokens: their masks and positions, and attention under them
over a 16-bit paged cache, against plain references (tests/tree_util.py)."""
import numpy as np
import pytest
import torch

from paged_util import attention as plain_attention
from paged_util import check_attention, make_step
from tree_util import attention, plan, random_parents

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    a.set_option(a.OPT_GRID_CTAS, 0)
    yield a
    a.set_option(a.OPT_GRID_CTAS, 0)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def starts(lens):
    return i32([0] + np.cumsum([n for _, n in lens]).tolist())


def flat(parents, pad=0):
    return i32([p for up in parents for p in up] + [7] * pad)


@pytest.mark.parametrize("lens,pad", [([(1, 1)], 0), ([(100, 16)], 3), ([(64, 64), (5, 5), (9, 0), (500, 63)], 0), ([(300, 65), (20, 7)], 70),
                                      ([(3, 7), (0, 2)], 1), ([(1000, 1 + i % 64) for i in range(1500)], 5)])
@pytest.mark.parametrize("with_positions", [True, False])
def test_plan(api, lens, pad, with_positions):
    rs = np.random.RandomState(len(lens) + pad)
    parents = [random_parents(rs, n) for _, n in lens]
    T = sum(n for _, n in lens) + pad
    masks, positions, ws = i64([5] * T), i32([5] * T) if with_positions else None, api.paged_workspace()
    api.tree_plan(flat(parents, pad), starts(lens), i32([s for s, _ in lens]), masks, positions, ws)
    assert api.last_launch_count() == 1 and api.read_status(ws) == 0
    want = plan(parents, lens)
    assert masks.tolist() == want[0] + [0] * pad
    if with_positions:
        assert positions.tolist() == want[1] + [-1] * pad


def test_plan_of_chains_and_stars(api):
    chain, star = list(range(-1, 63)), [-1] * 64
    masks, positions, ws = i64([0] * 128), i32([0] * 128), api.paged_workspace()
    api.tree_plan(flat([chain, star]), i32([0, 64, 128]), i32([70, 64]), masks, positions, ws)
    assert [m & (1 << 64) - 1 for m in masks.tolist()] == [(2 << i) - 1 for i in range(64)] + [1 << i for i in range(64)]
    assert positions.tolist() == list(range(6, 70)) + [0] * 64


@pytest.mark.parametrize("bad", [5, 3, -2, 64, 1 << 30, -(1 << 31)])
def test_plan_of_wrong_parents(api, bad):
    """Its own number, a later one and what is no token at all: reported, taken as a root."""
    masks, positions, ws = i64([0] * 5), i32([0] * 5), api.paged_workspace()
    api.tree_plan(i32([-1, 0, 1, bad, 3]), i32([0, 5]), i32([10]), masks, positions, ws)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    assert masks.tolist() == [1, 3, 7, 8, 24] and positions.tolist() == [5, 6, 7, 5, 6]


@pytest.mark.parametrize("q_start,seq", [([0, 2, -1], [5, 5]), ([0, 3, 2], [5, 5]), ([0, 9, 3], [5, 5]), ([-1, 2, 3], [5, 5]), ([0, 2, 900], [5, 5]), ([0, 2, 3], [-4, 5])])
def test_plan_of_wrong_requests(api, q_start, seq):
    """Rows of the request that is placed wrongly stay as they are."""
    masks, positions, ws = i64([9] * 4), i32([9] * 4), api.paged_workspace()
    api.tree_plan(i32([-1, 0, -1, 0]), i32(q_start), i32(seq), masks, positions, ws)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    if q_start in ([0, 2, -1], [0, 3, 2]):  # and what is padding is not known
        assert masks.tolist() == [1, 3] + ([9, 9] if q_start[1] == 2 else [4, 9])
    if q_start == [0, 2, 3]:
        assert masks.tolist() == [9, 9, 1, 0] and positions.tolist() == [9, 9, 4, -1]


def run(api, s, masks, lse=True, ws=None):
    q = s["q"]
    cache = api.KvCache(s["k"], s["v"])
    ws = api.paged_workspace(q.shape[1], cache) if ws is None else ws
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda") if lse else None
    api.paged_attention(q, cache, s["table"], s["q_start"], s["seq"], out, ws, lse=lse, tree_masks=masks)
    assert api.read_status(ws) == 0
    return out, lse


CASES = [
    # requests, page, heads, kv heads, d, type, layout
    ([(1001, 16)], 16, 32, 8, 128, torch.bfloat16, "bthd"),
    ([(16, 16), (17, 1), (40, 8), (0, 0), (129, 5)], 16, 8, 2, 64, torch.float16, "bhtd"),
    ([(300, 64), (64, 64), (190, 63), (1000, 33)], 48, 16, 4, 128, torch.bfloat16, "pair"),
    ([(128, 64), (129, 64), (192, 64), (65, 64), (260, 40)], 128, 4, 4, 64, torch.bfloat16, "bthd"),
    ([(700, 200), (333, 20), (90, 64), (5, 5)], 8, 8, 2, 128, torch.float16, "bthd"),
    ([(3, 7), (0, 2), (50, 50)], 16, 7, 1, 64, torch.bfloat16, "bthd"),
    ([(5000, 24)] * 3 + [(200, 64)] * 3, 64, 64, 4, 128, torch.bfloat16, "bthd"),
]


@pytest.mark.parametrize("lens,page,heads,kv,d,dtype,layout", CASES)
def test_attention(api, lens, page, heads, kv, d, dtype, layout):
    rs = np.random.RandomState(len(lens) * heads)
    s = make_step(lens, page, heads, kv, d, dtype, 3, layout, pad=2)
    masks = plan([random_parents(rs, n) for _, n in lens], lens)[0] + [0, 0]
    out, lse = run(api, s, i64(masks))
    check_attention(out, lse, attention(s, masks))
    again, _ = run(api, s, i64(masks), lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("ctas", [1, 7, 152])
def test_attention_under_any_masks(api, ctas):
    """Masks that are no tree's: rows that see nothing of the new tokens, not
    even themselves, bits of later tokens, a request without any context."""
    lens = [(64, 64), (20, 20), (200, 50), (7, 7)]
    s = make_step(lens, 16, 8, 2, 64, torch.bfloat16, 8)
    rs = np.random.RandomState(2)
    masks = [int(rs.randint(-(1 << 62), 1 << 62)) << 1 ^ int(rs.randint(0, 2)) for _ in range(141)]
    masks[0] = masks[3] = masks[64] = masks[134] = masks[140] = 0
    masks[100] = -1
    api.set_option(api.OPT_GRID_CTAS, ctas)
    out, lse = run(api, s, i64(masks))
    api.set_option(api.OPT_GRID_CTAS, 0)
    ref = attention(s, masks)
    assert (out[0] == 0).all() and lse[0].isneginf().all() and ref[1][0].isneginf().all()
    check_attention(out, lse, ref)


@pytest.mark.parametrize("lens,page,heads,kv,d,dtype,layout", CASES)
def test_chains_are_the_plain_call(api, lens, page, heads, kv, d, dtype, layout):
    """A tree without branches, and the plain call on the same inputs, against
    the same reference (their work is divided differently, so sums over keys are
    joined in other places)."""
    s = make_step(lens, page, heads, kv, d, dtype, 5, layout)
    masks = plan([list(range(-1, n - 1)) for _, n in lens], lens)[0]
    out, lse = run(api, s, i64(masks))
    cache = api.KvCache(s["k"], s["v"])
    ws, out2, lse2 = api.paged_workspace(heads, cache), torch.empty_like(out), torch.empty_like(lse)
    api.paged_attention(s["q"], cache, s["table"], s["q_start"], s["seq"], out2, ws, lse=lse2)
    ref = plain_attention(s)
    check_attention(out, lse, ref)
    check_attention(out2, lse2, ref)


def test_captured_and_replayed_at_other_trees(api):
    """The plan and two attentions that share a workspace, as one graph."""
    lens = [(300, 40), (90, 64), (20, 3)]
    T = 107
    s = make_step(lens, 16, 8, 2, 128, torch.bfloat16, 4)
    cache = api.KvCache(s["k"], s["v"])
    ws, parents, masks, positions = api.paged_workspace(8, cache), i32([-1] * T), i64([0] * T), i32([0] * T)
    outs = [torch.zeros_like(s["q"]) for _ in range(2)]

    def step():
        api.tree_plan(parents, s["q_start"], s["seq"], masks, positions, ws)
        for o in outs:
            api.paged_attention(s["q"], cache, s["table"], s["q_start"], s["seq"], o, ws, tree_masks=masks)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in (1, 2, 3):
            up = [random_parents(np.random.RandomState(seed), n) for _, n in lens]
            parents.copy_(flat(up))
            for o in outs:
                o.zero_()
            graph.replay()
            want = plan(up, lens)
            assert masks.tolist() == want[0] and positions.tolist() == want[1]
            check_attention(outs[0], None, attention(s, want[0]))
            assert torch.equal(outs[0], outs[1])
    torch.cuda.current_stream().wait_stream(stream)
    assert api.read_status(ws) == 0
