"""The paged step's plan, append and attention on the GPU against plain
64-bit references (tests/paged_util.py)."""
import math

import numpy as np
import pytest
import torch

from paged_util import attention, check_attention, make_cache, make_step

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan
def plan_reference(ctx, new, free, table, page, T, head=0):
    table, q0, taken = table.copy(), [0], 0
    slots, positions = np.full(T, -1), np.full(T, -1)
    for b, (c, n) in enumerate(zip(ctx, new)):
        for j in range(-(-c // page), min(-(-(c + n) // page), table.shape[1])):
            if head + taken < len(free):
                table[b, j] = free[head + taken]
                taken += 1
        for i in range(n):
            if q0[-1] + i < T:
                positions[q0[-1] + i] = c + i
                if (c + i) // page < table.shape[1] and table[b, (c + i) // page] >= 0:
                    slots[q0[-1] + i] = table[b, (c + i) // page] * page + (c + i) % page
        q0.append(q0[-1] + n)
    return table, q0, slots, positions, taken


def run_plan(api, ctx, new, free, table, page, T, head=None, with_positions=True):
    B = len(ctx)
    out = dict(q_start=i32([7] * (B + 1)), seq=i32([7] * B), slots=i32([7] * max(T, 1))[:T], taken=i32([7]),
               positions=i32([7] * max(T, 1))[:T] if with_positions else None, table=i32(table.tolist()))
    ws = api.paged_workspace()
    api.paged_plan(i32(ctx), i32(new), i32(free), out["table"], page, out["q_start"], out["seq"], out["slots"],
                   out["taken"], ws, positions=out["positions"], free_head=None if head is None else i32([head]))
    assert api.last_launch_count() == 1
    return out, api.read_status(ws)


def random_plan(B, page, seed, most_ctx, most_new, width):
    rs = np.random.RandomState(seed)
    ctx, new = rs.randint(0, most_ctx + 1, B).tolist(), rs.randint(0, most_new + 1, B).tolist()
    have = [-(-c // page) for c in ctx]
    order = rs.permutation(sum(have) + sum(-(-n // page) + 1 for n in new) + 5)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    return ctx, new, order[at:].tolist(), table


@pytest.mark.parametrize("B,page,most_ctx,most_new", [(1, 16, 0, 1), (1, 1, 40, 9), (3, 8, 100, 0), (16, 16, 900, 6),
                                                      (513, 48, 300, 40), (4096, 16, 64, 3)])
def test_plan(api, B, page, most_ctx, most_new):
    ctx, new, free, table = random_plan(B, page, B + page, most_ctx, most_new, (most_ctx + most_new) // page + 2)
    T = sum(new) + 5
    want = plan_reference(ctx, new, free, table, page, T)
    got, status = run_plan(api, ctx, new, free, table, page, T, with_positions=B != 3)
    assert status == 0
    assert got["table"].tolist() == want[0].tolist()
    assert got["q_start"].tolist() == want[1] and got["seq"].tolist() == [c + n for c, n in zip(ctx, new)]
    assert got["slots"].tolist() == want[2].tolist() and got["taken"].tolist() == [want[4]]
    if got["positions"] is not None:
        assert got["positions"].tolist() == want[3].tolist()


def test_plan_from_a_later_head_and_again(api):
    ctx, new, free, table = random_plan(9, 16, 3, 200, 60, 20)
    T = sum(new)
    want = plan_reference(ctx, new, free, table, 16, T, head=4)
    got, status = run_plan(api, ctx, new, free, table, 16, T, head=4)
    assert status == 0 and got["table"].tolist() == want[0].tolist() and got["slots"].tolist() == want[2].tolist()
    again, _ = run_plan(api, ctx, new, free, got["table"].cpu().numpy(), 16, T, head=4)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("short", ["tokens", "blocks", "width"])
def test_plan_out_of_room(api, short):
    ctx, new = [30, 5, 17], [10, 40, 3]
    table = np.full((3, 4 if short != "width" else 2), -1)
    table[0, :2], table[1, 0], table[2, :2] = [9, 8], 7, [6, 5]
    free = [0, 1, 2, 3, 4] if short != "blocks" else [0, 1]
    T = 53 if short != "tokens" else 20
    want = plan_reference(ctx, new, free, table, 16, T)
    got, status = run_plan(api, ctx, new, free, table, 16, T)
    assert status == api.EDEVICE_OVERFLOW
    assert got["table"].tolist() == want[0].tolist() and got["slots"].tolist() == want[2].tolist()
    assert got["taken"].tolist() == [want[4]] and got["q_start"].tolist() == [0, 10, 50, 53]


def test_plan_bad_lengths(api):
    got, status = run_plan(api, [-4, 3], [2, -7], [5, 6], np.array([[-1], [2]]), 16, 4)
    assert status == api.EDEVICE_BAD_INDEX
    assert got["q_start"].tolist() == [0, 2, 2] and got["slots"].tolist() == [80, 81, -1, -1]
    # the block that should hold the earlier tokens was never given
    got, status = run_plan(api, [3], [2], [5], np.array([[-1]]), 16, 2)
    assert status == api.EDEVICE_BAD_INDEX and got["slots"].tolist() == [-1, -1]


def test_plan_up_to_the_last_position(api):
    """A request near 2^31 tokens beside others: its position plus a token's
    place in the batch does not fit 32 bits."""
    page, width = 1024, 1 << 21
    ctx, new = [70, (1 << 31) - 1 - 1500, (1 << 31) - 1 - 900, 5], [1200, 1500, 700, 33]
    table = np.full((4, width), -1)
    table[0, 0], table[3, 0] = 3, 4
    for b in (1, 2):
        table[b, (ctx[b] - 1) // page] = 5 + b
    free, T = list(range(20, 40)), sum(new) + 4
    want = plan_reference(ctx, new, free, table, page, T)
    out = dict(q_start=i32([7] * 5), seq=i32([7] * 4), slots=i32([7] * T), taken=i32([7]), positions=i32([7] * T),
               table=torch.from_numpy(table.astype(np.int32)).cuda())
    ws = api.paged_workspace()
    api.paged_plan(i32(ctx), i32(new), i32(free), out["table"], page, out["q_start"], out["seq"], out["slots"], out["taken"], ws,
                   positions=out["positions"])
    assert api.read_status(ws) == 0
    assert (out["table"].cpu().numpy() == want[0]).all() and out["taken"].tolist() == [want[4]]
    assert out["slots"].tolist() == want[2].tolist() and out["positions"].tolist() == want[3].tolist()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("T,heads,d,page,dtype,layout", [(1, 1, 64, 8, torch.bfloat16, "bthd"), (37, 5, 128, 16, torch.float16, "bhtd"),
                                                         (515, 8, 128, 48, torch.bfloat16, "pair"), (2000, 2, 64, 24, torch.float16, "bthd")])
def test_append(api, T, heads, d, page, dtype, layout):
    n_blocks = T // page + 4
    k, v = make_cache(n_blocks, page, heads, d, dtype, T, layout)
    wk, wv = k.clone(), v.clone()
    fused = torch.randn((T, 3 * heads + 2, d), device="cuda").to(dtype)
    kn, vn = fused[:, 1:heads + 1], fused[:, 2 * heads + 1:3 * heads + 1]
    slots = torch.randperm(n_blocks * page, device="cuda")[:T].int()
    slots[T // 3:T // 3 + T // 10] = -1
    live = slots >= 0
    at = slots[live].long()
    wk[at // page, at % page] = kn[live]
    wv[at // page, at % page] = vn[live]
    ws = api.paged_workspace()
    api.paged_append(kn, vn, slots, api.KvCache(k, v), ws)
    assert api.read_status(ws) == 0
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_append_slots_outside_the_cache_are_skipped(api):
    k, v = make_cache(3, 16, 2, 64, torch.bfloat16, 1)
    wk = k.clone()
    kn = torch.randn((3, 2, 64), device="cuda").bfloat16()
    wk[0, 5] = kn[1]
    ws = api.paged_workspace()
    api.paged_append(kn, kn, i32([48, 5, -2]), api.KvCache(k, v), ws)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    assert torch.equal(k, wk)


# ------------------------------------------------------------------ attention
def run_attention(api, s, scale=0.0, lse=True, stream=None):
    cache = api.KvCache(s["k"], s["v"])
    ws = api.paged_workspace(s["q"].shape[1], cache)
    out = torch.full(s["q"].shape, math.nan, dtype=s["q"].dtype, device="cuda")
    z = torch.full(s["q"].shape[:2], math.nan, device="cuda") if lse else None
    api.paged_attention(s["q"], cache, s["table"], s["q_start"], s["seq"], out, ws, lse=z, scale=scale,
                        window=s["window"], stream=stream)
    assert api.read_status(ws) == 0
    return out, z


LENGTHS = {
    "one": [(1, 1)],
    "tile": [(128, 1), (129, 1), (127, 2), (256, 128)],
    "decode": [(1000, 1), (7, 1), (130, 1), (4097, 1), (64, 1)],
    "verify": [(611, 6), (6, 6), (2000, 3), (135, 16), (90, 1)],
    "chunk": [(300, 300), (777, 129), (40, 33)],
    "mixed": [(900, 200), (1, 1), (0, 0), (333, 5), (2049, 1)],
    "empty_rows": [(3, 7), (0, 2), (0, 0), (150, 160), (64, 1)],
}


@pytest.mark.parametrize("heads,kv_heads,d", [(4, 4, 64), (8, 2, 128), (14, 2, 64), (16, 1, 128), (15, 5, 128), (32, 1, 64)])
@pytest.mark.parametrize("lens", list(LENGTHS))
def test_attention_lengths_and_heads(api, lens, heads, kv_heads, d):
    dtype = torch.bfloat16 if (heads + len(lens)) % 2 else torch.float16
    s = make_step(LENGTHS[lens], 16, heads, kv_heads, d, dtype, heads + len(lens), pad=3)
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))
    assert (out[-3:] == 0).all() and (lse[-3:] == -math.inf).all()


@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 136, 256, 1024])
@pytest.mark.parametrize("layout", ["bthd", "bhtd", "pair"])
def test_attention_pages_and_layouts(api, page, layout):
    s = make_step([(1500, 5), (page, 1), (page + 1, 2), (700, 150)], page, 8, 2, 64 if page % 48 else 128, torch.bfloat16, page, layout=layout)
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 5000])
@pytest.mark.parametrize("page", [16, 136])
def test_attention_window(api, window, page):
    s = make_step([(1500, 1), (1300, 6), (900, 250), (3, 2)], page, 8, 2, 128, torch.float16, window, window=window)
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))


@pytest.mark.parametrize("grid", [1, 2, 7, 61])
@pytest.mark.parametrize("lens", ["decode", "mixed", "empty_rows"])
def test_attention_on_other_grids(api, grid, lens):
    """The division over the CTAs, and so the joining of parts, is another."""
    s = make_step(LENGTHS[lens], 32, 12, 4, 128, torch.bfloat16, grid)
    api.set_option(api.OPT_GRID_CTAS, grid)
    try:
        out, lse = run_attention(api, s)
    finally:
        api.set_option(api.OPT_GRID_CTAS, 0)
    check_attention(out, lse, attention(s))


def test_attention_many_requests(api):
    rs = np.random.RandomState(5)
    lens = [(int(s), int(min(n, s))) for s, n in zip(rs.randint(0, 400, 700), rs.randint(0, 4, 700))]
    s = make_step(lens, 16, 4, 2, 64, torch.bfloat16, 5)
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))


@pytest.mark.parametrize("lens", ["verify", "chunk"])
def test_attention_strided_queries_scale_and_no_lse(api, lens):
    s = make_step(LENGTHS[lens], 16, 8, 2, 64, torch.bfloat16, 11)
    T = s["q"].shape[0]
    fused = torch.zeros((T, 12, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = s["q"]
    s["q"] = fused[:, 2:10]
    out, _ = run_attention(api, s, scale=0.31, lse=False)
    check_attention(out, None, attention(s, scale=0.31))
    # heads outermost
    s["q"] = s["q"].transpose(0, 1).contiguous().transpose(0, 1)
    again, _ = run_attention(api, s, scale=0.31)
    assert torch.equal(out, again)


@pytest.mark.parametrize("lens", ["verify", "chunk"])
def test_attention_large_scores(api, lens):
    """Scores of some hundreds: one key takes nearly all the weight, and the
    running maximum moves by more than fp32's exponent can undo."""
    s = make_step(LENGTHS[lens], 16, 8, 2, 128, torch.bfloat16, 12)
    s["q"] *= 25
    out, lse = run_attention(api, s)
    o, z, mag = attention(s)
    # a score of 400 carries an error of 400 * 128 * 2^-24 in the worst case,
    # which is the relative error of its weight
    err = (out.double() - o).abs()
    assert (err <= (2.0 ** -7 + 2.0 ** -8) * mag).all()
    assert ((lse.double() - z).abs() <= 2.0 ** -8).all()


def test_attention_is_deterministic_and_repeats(api):
    s = make_step(LENGTHS["mixed"], 16, 8, 2, 128, torch.bfloat16, 13)
    a, za = run_attention(api, s)
    for _ in range(3):
        b, zb = run_attention(api, s)
        assert torch.equal(a, b) and torch.equal(za, zb)


def test_attention_offsets_beyond_32_bits(api):
    """A cache of more than 2^31 elements in each of K and V."""
    page, kv, d = 16, 8, 128
    n_blocks = (1 << 31) // (page * kv * d) + 64
    k = torch.zeros((n_blocks, page, kv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    lens, table = [(75, 2)], np.array([[n_blocks - 1, n_blocks - 3, 1, n_blocks - 7, n_blocks - 20]], np.int32)
    for b in table[0]:
        k[int(b)].normal_()
        v[int(b)].normal_()
    q = torch.randn((2, 16, d), device="cuda").bfloat16()
    s = dict(q=q, k=k, v=v, table=torch.from_numpy(table).cuda(), q_start=i32([0, 2]), seq=i32([75]), lens=lens, window=0)
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))
    new = torch.randn((1, kv, d), device="cuda").bfloat16()
    ws = api.paged_workspace()
    api.paged_append(new, new, i32([(n_blocks - 1) * page + 3]), api.KvCache(k, v), ws)
    assert api.read_status(ws) == 0 and torch.equal(k[n_blocks - 1, 3], new[0]) and torch.equal(v[n_blocks - 1, 3], new[0])
    del k, v, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("what", ["block", "width", "q_start", "seq"])
def test_attention_bad_tables_are_reported(api, what):
    """The kernel checks every block number, the table's width and the
    lengths before it uses them; other requests' rows are right."""
    s = make_step([(200, 2), (300, 1)], 16, 4, 2, 64, torch.bfloat16, 17)
    want = attention(s)
    table, q_start, seq = s["table"].clone(), s["q_start"].clone(), s["seq"].clone()
    if what == "block":
        table[0, 3], table[0, 5] = 1 << 30, -5
    elif what == "width":
        seq[0] = 16 * table.shape[1] + 9
    elif what == "q_start":
        q_start[0] = -3
    else:
        seq[0] = -1
    cache = api.KvCache(s["k"], s["v"])
    ws = api.paged_workspace(4, cache)
    out = torch.zeros_like(s["q"])
    api.paged_attention(s["q"], cache, table, q_start, seq, out, ws)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    check_attention(out[2:], None, [t[2:] for t in want])


def test_step_on_a_side_stream_and_in_a_graph(api):
    """Plan, append and attention of a step, captured: replays follow the
    lengths in the device buffers."""
    page, kv, heads, d, B, T = 16, 2, 8, 64, 3, 12
    k, v = make_cache(64, page, kv, d, torch.bfloat16, 21)
    k.zero_(), v.zero_()
    cache = api.KvCache(k, v)
    ws, wa = api.paged_workspace(), api.paged_workspace(heads, cache)
    ctx, new = i32([0, 0, 0]), i32([4, 2, 0])
    free, head = torch.randperm(64, device="cuda").int(), i32([0])
    table, q_start, seq = i32([[-1] * 8] * B), i32([0] * (B + 1)), i32([0] * B)
    slots, taken = i32([0] * T), i32([0])
    q, kn, vn = (torch.empty((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (heads, kv, kv))
    out, lse = torch.empty_like(q), torch.empty((T, heads), device="cuda")

    def step():
        api.paged_plan(ctx, new, free, table, page, q_start, seq, slots, taken, ws, free_head=head)
        api.paged_append(kn, vn, slots, cache, ws)
        api.paged_attention(q, cache, table, q_start, seq, out, wa, lse=lse)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    past_k, past_v = [[] for _ in range(B)], [[] for _ in range(B)]
    for it, lens in enumerate([[4, 2, 0], [1, 6, 5], [3, 0, 1], [9, 2, 1], [1, 1, 1], [6, 6, 0]]):
        new.copy_(i32(lens))
        for t in (q, kn, vn):
            t.normal_()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            if it % 2:
                step()
            else:
                graph.replay()
        torch.cuda.default_stream().wait_stream(side)
        at = 0
        for b, n in enumerate(lens):
            past_k[b].append(kn[at:at + n].clone())
            past_v[b].append(vn[at:at + n].clone())
            at += n
        assert api.read_status(ws) == 0 and api.read_status(wa) == 0
        at = 0
        for b, n in enumerate(lens):
            kk, vv = torch.cat(past_k[b]), torch.cat(past_v[b])
            if n:
                flat = dict(q=q[at:at + n], k=kk[:, None], v=vv[:, None], window=0, lens=[(len(kk), n)],
                            table=torch.arange(len(kk), device="cuda").int()[None])
                ref = attention(flat)
                check_attention(out[at:at + n], lse[at:at + n], ref, (it, b))
            at += n
        ctx.copy_(seq)
        head += taken


@pytest.mark.parametrize("heads,kv_heads,d", [(8, 1, 128), (64, 8, 64), (14, 2, 128)])
@pytest.mark.parametrize("new", [9, 10, 12, 16, 18])
@pytest.mark.parametrize("grid", [0, 3])
def test_attention_around_one_slots_rows(api, heads, kv_heads, d, new, grid):
    """Some 64 to 128 rows a kv head: items of one slot and of both of the chunk
    kernel, of one tile, of two and of many, next to each other."""
    lens = [(new, new), (1500, new), (128 + new, new), (127, new), (2000, 3 * new), (129, new), (700, new)]
    s = make_step(lens, 16, heads, kv_heads, d, torch.bfloat16, new, window=0 if new % 4 else 300)
    api.set_option(api.OPT_GRID_CTAS, grid)
    try:
        out, lse = run_attention(api, s)
    finally:
        api.set_option(api.OPT_GRID_CTAS, 0)
    check_attention(out, lse, attention(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("below", [10, 23, 25, 27, 33])
def test_attention_to_many_keys_far_below_one(api, dtype, new, below):
    """One key takes nearly all the weight, the others 2^-below of it each, but
    there are many: what they add has to be there to the type's rounding, also
    where a weight of 2^-25 is less than fp16 has next to 1."""
    seq, d = 60000, 64
    s = make_step([(seq, new)], 16, 4, 2, d, dtype, 31, poison=False)
    s["q"].fill_(0.5)
    s["k"].zero_()
    s["v"].fill_(1.0)
    first = int(s["table"][0, 0])
    # q.k / sqrt(d) = 64 * 0.5 * x / 8 = 4 x, in nats
    s["k"][first, 3] = below * math.log(2) / 4
    s["v"][first, 3] = 0.0
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))


@pytest.mark.parametrize("grid", [0, 1, 61])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_to_a_nan_key(api, d, grid):
    """Rows that see a NaN score are NaN, in lse too (-inf would say that they
    see nothing); the rows before it and the other heads are as without it."""
    s = make_step([(1000, 1), (2000, 6), (900, 300), (333, 20)], 16, 8, 2, d, torch.bfloat16, d)
    api.set_option(api.OPT_GRID_CTAS, grid)
    try:
        out, lse = run_attention(api, s)
        hit = torch.zeros_like(lse, dtype=torch.bool)
        table, t0 = s["table"].cpu(), 0
        for b, (seq, n) in enumerate(s["lens"]):
            key = seq - (n + 1) // 2
            s["k"][int(table[b, key // 16]), key % 16, 1] = math.nan
            hit[t0 + n - (n + 1) // 2:t0 + n, 4:] = True
            t0 += n
        got, z = run_attention(api, s)
    finally:
        api.set_option(api.OPT_GRID_CTAS, 0)
    assert got[hit].isnan().all() and z[hit].isnan().all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(z[~hit], lse[~hit])


@pytest.mark.parametrize("window", [1 << 28, 1 << 30, (1 << 31) - 2, (1 << 31) - 1])
@pytest.mark.parametrize("lens", ["empty_rows", "decode", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_windows_wider_than_everything(api, lens, window, d):
    """Next to rows at negative positions too, a window of any size counts back
    from each row's position."""
    s = make_step(LENGTHS[lens], 16, 8, 2, d, torch.bfloat16, 41, window=window, pad=1)
    out, lse = run_attention(api, s)
    check_attention(out, lse, attention(s))


@pytest.mark.parametrize("new", [1, 6, 20, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("short", [0, 1, 33, 127, 128, 1000])
def test_attention_up_to_the_last_position(api, new, d, short):
    """Positions up to 2^31 - 2 under a window: the keys' numbers, rounded up to
    whole tiles, do not fit 32 bits. The same as a short request's, moved by whole
    pages."""
    page, window, near = 1024, 500, 4 * 1024 - 1 - short
    s = make_step([(near, new)], page, 8, 2, d, torch.bfloat16, 43, window=window, width=4)
    want = attention(s)
    moved = (1 << 31) - 4 * page
    table = torch.full((1, 1 << 21), -1, dtype=torch.int32, device="cuda")
    table[0, -4:] = s["table"][0]
    s["table"], s["seq"] = table, i32([near + moved])
    out, lse = run_attention(api, s)
    check_attention(out, lse, want)


@pytest.mark.parametrize("lens", list(LENGTHS))
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 128), (32, 1, 64)])
def test_attention_waits_that_run_out(api, lens, heads, kv_heads, d):
    """Keys that never come: the call ends, reports it, and leaves nothing behind
    that still writes where the next call works. The next ones follow at once on
    the same SMs, on a workspace of their own; the call's own serves again once it
    is initialised."""
    s = make_step(LENGTHS[lens], 16, heads, kv_heads, d, torch.bfloat16, 47)
    cache = api.KvCache(s["k"], s["v"])
    ws, other = api.paged_workspace(heads, cache), api.paged_workspace(heads, cache)
    outs = [torch.full_like(s["q"], math.nan) for _ in range(5)]

    def call(out, ws):
        api.paged_attention(s["q"], cache, s["table"], s["q_start"], s["seq"], out, ws)

    torch.cuda.synchronize()
    api.set_option(api.OPT_WAIT_TIMEOUT_NS, 2_000_000)
    api.set_option(api.OPT_DEBUG_HOLD_BACK, 1)
    try:
        call(outs[0], ws)
    finally:
        api.set_option(api.OPT_DEBUG_HOLD_BACK, 0)
        api.set_option(api.OPT_WAIT_TIMEOUT_NS, 1_000_000_000)
    for out in outs[1:4]:
        call(out, other)
    assert api.read_status(ws) == api.ETIMEOUT
    api.workspace_init(ws)
    call(outs[4], ws)
    assert api.read_status(ws) == 0 and api.read_status(other) == 0
    want = attention(s)
    for out in outs[1:]:
        check_attention(out, None, want)


@pytest.mark.parametrize("what", ["seq", "past_T"])
def test_attention_requests_that_do_not_fit_are_left_out(api, what):
    """Their rows keep what was there; the others' are right."""
    s = make_step([(200, 2), (300, 90), (77, 3)], 16, 4, 2, 64, torch.bfloat16, 53)
    want = attention(s)
    q_start, seq = s["q_start"].clone(), s["seq"].clone()
    good = torch.ones(95, dtype=torch.bool, device="cuda")
    if what == "seq":
        seq[1] = -5
        good[2:92] = False
    else:
        q_start[3] = 96
        good[92:] = False
    cache = api.KvCache(s["k"], s["v"])
    ws = api.paged_workspace(4, cache)
    out, lse = torch.full_like(s["q"], 7.0), torch.full(s["q"].shape[:2], 7.0, device="cuda")
    api.paged_attention(s["q"], cache, s["table"], q_start, seq, out, ws, lse=lse)
    assert api.read_status(ws) == api.EDEVICE_BAD_INDEX
    assert (out[~good] == 7).all() and (lse[~good] == 7).all()
    check_attention(out[good], lse[good], [t[good] for t in want])


def test_one_token_of_an_odd_width(api):
    """One request's one token, sliced out of a projection whose width is not a
    multiple of 8."""
    page, heads, d = 16, 8, 64
    s = make_step([(100, 1)], page, heads, 1, d, torch.bfloat16, 59, poison=False)
    width = (heads + 2) * d + 3
    rows = torch.randn((1, width), device="cuda").bfloat16().as_strided((1, heads + 2, d), (width, d, 1))
    cache, ws = api.KvCache(s["k"], s["v"]), api.paged_workspace(heads, api.KvCache(s["k"], s["v"]))
    out = torch.empty((1, heads, d), dtype=torch.bfloat16, device="cuda")
    slot = s["table"][:, 99 // page] * page + 99 % page
    api.paged_append(rows[:, heads:heads + 1], rows[:, heads + 1:], slot.int(), cache, ws)
    api.paged_attention(rows[:, :heads], cache, s["table"], s["q_start"], s["seq"], out, ws)
    assert api.read_status(ws) == 0
    assert torch.equal(s["k"][int(s["table"][0, 6]), 3], rows[0, heads:heads + 1])
    s["q"] = rows[:, :heads].contiguous()
    check_attention(out, None, attention(s))
