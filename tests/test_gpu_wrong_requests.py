"""Requests that q_start or seq_lens place wrongly: reported, their rows left as
they were, the other requests' as in a call without them, and no padding rows
where the last request is the wrong one (where they begin is not known)."""
import pytest
import torch

import paged_util
from cache8_util import make_step8

pytestmark = pytest.mark.gpu

# q_start, seq_lens, rows of the valid requests, padding rows (of four rows)
WRONG = [
    ([0, 2, -1], [5, 5], [0, 1], []),
    ([0, 3, 2], [5, 5], [0, 1, 2], []),
    ([0, 9, 3], [5, 5], [], []),
    ([-1, 2, 3], [5, 5], [2], [3]),
    ([0, 2, 900], [5, 5], [0, 1], []),
    ([0, 2, 3], [-4, 5], [2], [3]),
    ([0, 1, 3], [5, -1], [0], [3]),
]


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    a.set_option(a.OPT_GRID_CTAS, 0)
    return a


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("q_start,seq,masks,positions", [
    ([0, 2, -1], [5, 5], [1, 3, 9, 9], [3, 4, 9, 9]), ([0, 3, 2], [5, 5], [1, 3, 4, 9], [2, 3, 2, 9]),
    ([0, 9, 3], [5, 5], [9, 9, 9, 9], [9, 9, 9, 9]), ([-1, 2, 3], [5, 5], [9, 9, 1, 0], [9, 9, 4, -1]),
    ([0, 2, 900], [5, 5], [1, 3, 9, 9], [3, 4, 9, 9]), ([0, 2, 3], [-4, 5], [9, 9, 1, 0], [9, 9, 4, -1]),
    ([0, 1, 3], [5, -1], [1, 9, 9, 0], [4, 9, 9, -1])])
def test_tree_plan(api, q_start, seq, masks, positions):
    got, at, ws = torch.full((4,), 9, dtype=torch.int64, device="cuda"), i32([9] * 4), api.paged_workspace()
    api.tree_plan(i32([-1, 0, -1, 0]), i32(q_start), i32(seq), got, at, ws)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    assert got.tolist() == masks and at.tolist() == positions


@pytest.mark.parametrize("q_start,seq,rows,padding", WRONG)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("codes", [False, True])
def test_attention(api, codes, tree, q_start, seq, rows, padding):
    """Each valid request's rows bit for bit as by a call of it alone."""
    heads, kv = 8, 2
    if codes:
        s = make_step8(api, [(5, 2), (5, 2)], 16, heads, kv, 64, torch.bfloat16, 3)
        cache = s["cache"]
    else:
        s = paged_util.make_step([(5, 2), (5, 2)], 16, heads, kv, 64, torch.bfloat16, 3)
        cache = api.KvCache(s["k"], s["v"])
    masks = torch.full((4,), -1, dtype=torch.int64, device="cuda") if tree else None
    ws = api.paged_workspace(heads, cache)

    def call(table, q_start, seq, T=4):
        out, lse = torch.full((T, heads, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, heads), 3.0, device="cuda")
        api.paged_attention(s["q"][:T], cache, table, i32(q_start), i32(seq), out, ws, lse=lse, tree_masks=None if masks is None else masks[:T])
        return out, lse

    want, want_lse = torch.full((4, heads, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, heads), 3.0, device="cuda")
    for b in range(2):
        if rows and q_start[b] <= rows[0] < q_start[b + 1]:
            one, one_lse = call(s["table"][b:b + 1], [rows[0], rows[-1] + 1], [seq[b]])
            want[rows], want_lse[rows] = one[rows], one_lse[rows]
    want[padding], want_lse[padding] = 0.0, -float("inf")
    api.workspace_init(ws)
    out, lse = call(s["table"], q_start, seq)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
