"""Attention over a paged cache of 8-bit values against plain 64-bit references
(tests/cache8_util.py, tests/paged_util.py, tests/tree_util.py)."""
import math

import numpy as np
import pytest
import torch

import paged_util
import tree_util
from cache8_util import check_attention8, make_step8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    a.set_option(a.OPT_GRID_CTAS, 0)
    a.set_option(a.OPT_WAIT_TIMEOUT_NS, 1_000_000_000)
    yield a
    a.set_option(a.OPT_GRID_CTAS, 0)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def run(api, s, masks=None, lse=True, ws=None, status=0, **kw):
    q = s["q"]
    ws = api.paged_workspace(q.shape[1], s["cache"]) if ws is None else ws
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda") if lse else None
    api.paged_attention(q, s["cache"], s["table"], s["q_start"], s["seq"], out, ws, lse=lse, window=s["window"], tree_masks=masks, **kw)
    assert api.last_launch_count() == 1 and api.read_status(ws) == status
    return out, lse


CASES = [
    # requests, page, heads, kv heads, d, type, layout, window
    ([(1, 1)], 16, 1, 1, 64, torch.bfloat16, "bthd", 0),
    ([(1001, 1)], 16, 32, 8, 128, torch.bfloat16, "bthd", 0),
    ([(5, 1), (128, 1), (129, 1), (127, 2), (0, 0), (256, 16)], 16, 8, 2, 64, torch.float16, "bhtd", 0),
    ([(16, 16), (17, 6), (2500, 6), (300, 5)], 48, 28, 4, 128, torch.bfloat16, "pair", 0),
    ([(700, 200), (1, 1), (333, 5), (2049, 1)], 32, 8, 2, 128, torch.float16, "bthd", 0),
    ([(300, 100), (64, 64)], 128, 16, 16, 64, torch.bfloat16, "bthd", 0),
    ([(3, 7), (0, 2), (150, 160)], 16, 7, 1, 128, torch.bfloat16, "bthd", 0),
    ([(900, 4), (50, 20), (1300, 33)], 64, 8, 1, 64, torch.float16, "bhtd", 100),
    ([(900, 4), (50, 20), (1300, 33)], 1024, 32, 1, 128, torch.bfloat16, "bthd", 1),
    ([(20000, 1)], 16, 64, 8, 128, torch.float16, "bthd", 0),
    ([(700, 6)] * 40, 16, 32, 8, 128, torch.bfloat16, "bthd", 0),
    ([(40 + 13 * i, 1) for i in range(65)], 112, 6, 3, 64, torch.bfloat16, "pair", 0),
]


@pytest.mark.parametrize("lens,page,heads,kv,d,dtype,layout,window", CASES)
def test_attention(api, lens, page, heads, kv, d, dtype, layout, window):
    s = make_step8(api, lens, page, heads, kv, d, dtype, 3, layout, window, pad=2)
    out, lse = run(api, s)
    ref = paged_util.attention(s)
    check_attention8(out, lse, ref, max(n for n, _ in lens))
    again, _ = run(api, s, lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("ctas", [1, 3, 61])
def test_on_other_grids(api, ctas):
    lens = [(900, 200), (1, 1), (0, 0), (333, 5), (2049, 1)]
    s = make_step8(api, lens, 16, 8, 2, 128, torch.bfloat16, 5)
    api.set_option(api.OPT_GRID_CTAS, ctas)
    out, lse = run(api, s)
    api.set_option(api.OPT_GRID_CTAS, 0)
    check_attention8(out, lse, paged_util.attention(s), 2049)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_of_very_different_sizes(api, d, dtype):
    """Powers of two of the values from 2^-30 (fp16: 2^-8) to 2^30 (2^8) token by
    token: a row that sees small ones alone has as many bits as any."""
    by = 30 if dtype == torch.bfloat16 else 8
    lens = [(40, 40), (400, 30), (1000, 3)]
    s = make_step8(api, lens, 16, 4, 2, d, dtype, 6, spread=(0.5, 0.0))
    rs = np.random.RandomState(9)
    e = torch.from_numpy(rs.randint(-by, by + 1, s["cache"].v_scale.shape)).cuda()
    first = s["table"][0, 0]
    e[first, :, 0], e[first, :, 1:] = -by, by  # the first token small, those after it large
    real = s["cache"].v_scale != 255
    s["cache"].v_scale[real] = (s["cache"].v_scale[real].int() + e[real].int()).to(torch.uint8)
    s["v"] = s["v"] * torch.exp2(e.double()).transpose(1, 2)[..., None]
    out, lse = run(api, s)
    check_attention8(out, lse, paged_util.attention(s), 1000)


def test_queries_and_keys_of_very_different_sizes(api):
    """Rows of queries from 2^-40 to 2^40 against keys of 2^40 down to 2^-40:
    the scores are of usual size."""
    lens = [(300, 20)]
    s = make_step8(api, lens, 16, 8, 8, 64, torch.bfloat16, 7, spread=(0.5, 0.5))
    e = torch.tensor([-40, -20, -7, 0, 1, 13, 30, 40], device="cuda")  # by head
    s["q"] = (s["q"].float() * torch.exp2(e.float())[None, :, None]).bfloat16()
    real = s["cache"].k_scale != 255
    s["cache"].k_scale.copy_(torch.where(real, (s["cache"].k_scale.int() - e.int()[None, :, None]).to(torch.uint8), s["cache"].k_scale))
    s["k"] = s["k"] * torch.exp2(-e.double())[None, None, :, None]
    out, lse = run(api, s)
    check_attention8(out, lse, paged_util.attention(s), 300)


@pytest.mark.parametrize("scale", [0.01, 3.0])
def test_scale(api, scale):
    s = make_step8(api, [(500, 7), (60, 60)], 32, 8, 2, 128, torch.float16, 8, spread=(0.3, 0.3))
    out, lse = run(api, s, scale=scale)
    ref = paged_util.attention(s, scale)
    # the scores, of up to some 3 * 11 * 30, are off by their products' rounding: 2^-24 of the magnitudes' sum a term
    check_attention8(out, None, ref, 500)
    assert ((lse.double() - ref[1]).abs() <= 2.0 ** -13 + 2.0 ** -20 * ref[1].abs()).all()


def test_what_is_not_a_number(api):
    """A key's or a value's byte of 255 reaches the rows that see it; other heads
    and requests are as they were."""
    lens = [(100, 10), (100, 10)]
    s = make_step8(api, lens, 16, 8, 2, 64, torch.bfloat16, 9)
    want, want_lse = run(api, s)
    for scale, lse_too in ((s["cache"].k_scale, True), (s["cache"].v_scale, False)):
        at = s["table"][0, 3], 1, 5  # token 53 of request 0, kv head 1
        was = scale[at].item()
        scale[at] = 255
        out, lse = run(api, s)
        assert out[:10, 4:].isnan().all() and torch.equal(out[:10, :4], want[:10, :4]) and torch.equal(out[10:], want[10:])
        assert lse[:10, 4:].isnan().all() if lse_too else torch.equal(lse, want_lse)
        scale[at] = was
    s["q"][3, 2, 7] = math.nan
    out, lse = run(api, s)
    assert out[3, 2].isnan().all() and lse[3, 2].isnan() and torch.equal(out[4:], want[4:]) and torch.equal(out[:3], want[:3])


def test_bad_tables_and_requests_are_reported(api):
    lens = [(100, 10), (90, 4)]
    s = make_step8(api, lens, 16, 8, 2, 64, torch.bfloat16, 10)
    want, _ = run(api, s)
    table = s["table"].clone()
    for bad in (-1, 10 ** 6):
        s["table"] = table.clone()
        s["table"][0, 2] = bad
        out, _ = run(api, s, status=api.EDEVICE_BAD_INDEX)
        assert torch.equal(out[10:], want[10:])
    s["table"] = table[:, :5].contiguous()  # the last keys beyond the table
    out, _ = run(api, s, status=api.EDEVICE_BAD_INDEX)
    s["table"], seq = table, s["seq"].clone()
    s["seq"] = torch.tensor([-3, 90], dtype=torch.int32, device="cuda")
    out, _ = run(api, s, status=api.EDEVICE_BAD_INDEX)
    assert torch.equal(out[10:], want[10:]) and (out[:10] == 3.0).all()
    s["seq"] = seq


TREES = [
    ([(1001, 16)], 16, 32, 8, 128, torch.bfloat16),
    ([(16, 16), (17, 1), (40, 8), (0, 0), (129, 5), (300, 64)], 16, 8, 2, 64, torch.float16),
    ([(300, 64), (64, 64), (190, 63), (400, 80)], 48, 16, 4, 128, torch.bfloat16),
    ([(3, 7), (50, 50)], 128, 4, 4, 64, torch.bfloat16),
]


@pytest.mark.parametrize("lens,page,heads,kv,d,dtype", TREES)
def test_trees(api, lens, page, heads, kv, d, dtype):
    rs = np.random.RandomState(len(lens) * heads)
    s = make_step8(api, lens, page, heads, kv, d, dtype, 11, pad=3)
    masks = tree_util.plan([tree_util.random_parents(rs, n) for _, n in lens], lens)[0] + [0, 0, 0]
    out, lse = run(api, s, i64(masks))
    check_attention8(out, lse, tree_util.attention(s, masks), max(n for n, _ in lens))
    chain = tree_util.plan([list(range(-1, n - 1)) for _, n in lens], lens)[0] + [0, 0, 0]
    a, b = run(api, s, i64(chain)), run(api, s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_trees_under_any_masks(api):
    lens = [(64, 64), (20, 20), (200, 50), (7, 7)]
    s = make_step8(api, lens, 16, 8, 2, 64, torch.bfloat16, 12)
    rs = np.random.RandomState(2)
    masks = [int(rs.randint(-(1 << 62), 1 << 62)) << 1 ^ int(rs.randint(0, 2)) for _ in range(141)]
    masks[0] = masks[3] = masks[64] = masks[134] = masks[140] = 0
    out, lse = run(api, s, i64(masks))
    assert (out[0] == 0).all() and lse[0].isneginf().all()
    check_attention8(out, lse, tree_util.attention(s, masks), 200)


def test_with_masks_there_is_no_window(api):
    s = make_step8(api, [(20, 4)], 16, 8, 2, 64, torch.bfloat16, 12, window=5)
    with pytest.raises(api.MoeError):
        run(api, s, i64([0] * 4))


def test_waits_that_run_out(api):
    """The first keys of each CTA never come: the waits end, the status says so,
    calls on the workspace are right again once it is zeroed."""
    s = make_step8(api, [(300, 3)] * 4, 16, 8, 2, 128, torch.bfloat16, 13)
    ws = api.paged_workspace(8, s["cache"])
    api.set_option(api.OPT_DEBUG_HOLD_BACK, 1)
    api.set_option(api.OPT_WAIT_TIMEOUT_NS, 2_000_000)
    try:
        run(api, s, ws=ws, status=api.ETIMEOUT)
    finally:
        api.set_option(api.OPT_DEBUG_HOLD_BACK, 0)
        api.set_option(api.OPT_WAIT_TIMEOUT_NS, 1_000_000_000)
    api.workspace_init(ws)
    out, lse = run(api, s, ws=ws)
    check_attention8(out, lse, paged_util.attention(s), 300)


def test_captured_and_replayed_at_other_lengths(api):
    lens = [(300, 6), (90, 6), (20, 6)]
    s = make_step8(api, lens, 16, 8, 2, 128, torch.bfloat16, 14)
    ws, out = api.paged_workspace(8, s["cache"]), torch.zeros_like(s["q"])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            api.paged_attention(s["q"], s["cache"], s["table"], s["q_start"], s["seq"], out, ws)
        for seqs in ((300, 90, 20), (250, 6, 19), (7, 81, 6)):
            s["seq"].copy_(torch.tensor(seqs, dtype=torch.int32))
            s["lens"] = [(n, 6) for n in seqs]
            out.zero_()
            graph.replay()
            check_attention8(out, None, paged_util.attention(s), 300)
    torch.cuda.current_stream().wait_stream(stream)
    assert api.read_status(ws) == 0


def test_far_into_a_large_cache(api):
    """Slots beyond 2^31 bytes of codes: written, rotated, read back and attended
    over as at the beginning."""
    heads, page, d, n_blocks = 8, 16, 128, 140000  # 2.3 GB of K, and of V
    k, v = (torch.empty((n_blocks, page, heads, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((n_blocks, heads, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = api.KvCache8(k, v, ks, vs)
    x = torch.randn((2, 40, heads, d), device="cuda").bfloat16()
    positions, r = torch.arange(40, device="cuda").int(), api.Rope(d)
    q = torch.randn((2, 32, d), device="cuda").bfloat16()
    ws, got = api.paged_workspace(32, cache), []
    for blocks in ([0, 2, 5], [n_blocks - 1, n_blocks - 2, n_blocks - 7]):
        table = torch.tensor([blocks], dtype=torch.int32, device="cuda")
        slots = (table[0].long()[positions.long() // page] * page + positions % page).int()
        back, out = torch.empty_like(x), torch.empty_like(q)
        api.paged_rope_append(None, x[0], x[1], positions, slots, r, cache, ws)
        api.paged_read(cache, slots, back[0], back[1], ws)
        starts, seq = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
        api.paged_attention(q, cache, table, starts, seq, out, ws)
        got.append((back, out))
    assert api.read_status(ws) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert ((got[0][0][1].double() - x[1].double()).abs() <= 2.0 ** -4 * x[1].double().abs() + 2.0 ** -10 * x[1].double().abs().amax(-1, keepdim=True) / 224).all()
