"""The operators of a decode, speculative-verify or chunked-prompt step around the MoE layer, as they are measured: the step's plan
(block tables and slot maps from request lengths), the write of new keys and values into a paged cache, the attention of the new
tokens over that cache, and sampling from the output layer's logits.

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes one pass (the plain form in
elementary torch operations, or the library's calls where ``own`` is true), ``exact`` gives the same outputs from the definitions in
64 bits.
"""
import math

import numpy as np
import torch

own = False

VOCAB = 157184  # rows of the output layer that the benchmark measures


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one stream, one new token, a short history: latency is all there is
        attn("attn_decode_short", 1, "1", "1000", 32, 8, 128, 16, "bf16", 0),
        # 32 streams verifying chains of 6 speculated tokens, histories of all lengths
        attn("attn_verify_batch", 32, "6", "300-16000", 32, 8, 128, 16, "bf16", 0),
        # a few streams deep into long documents, one token each: the cache's bandwidth
        attn("attn_decode_long", 4, "1", "120001-131070", 64, 8, 128, 64, "f16", 0),
        # two prompts taken in chunks of 8192, the second chunk: matrix products
        attn("attn_chunk_large", 2, "8192", "8191", 32, 8, 128, 32, "bf16", 0),
        # one prompt's chunk next to streams that decode, a sliding window, heads that share nothing, pages of 48
        attn("attn_mixed_window", 17, "first:515,1-6", "0-3500", 16, 16, 64, 48, "f16", 1024),
        # one token from the output layer's logits: latency
        sample("sample_one", 1, VOCAB, "f32"),
        # the largest verify block, other settings in each row
        sample("sample_block", 16, VOCAB, "f32"),
        # a serving batch over an odd vocabulary, 16-bit logits with their ties
        sample("sample_batch", 256, 50257, "bf16"),
        # the plan of a verify step of 16 streams
        plan("plan_verify", 16, "6", "100-8000", 16, 600),
        # the plan of a full step: chunks of prompts next to hundreds of decoding streams
        plan("plan_full", 512, "first:8191,1-64", "0-6000", 16, 2048),
        # the new keys and values of a verify step
        append("append_verify", 96, 8, 128, 16, 2048, "bf16"),
        # those of a full chunk
        append("append_chunk", 8192, 8, 128, 16, 8192, "bf16"),
    ]


def attn(name, B, new, ctx, hq, hkv, d, page, dtype, window):
    return {"name": name, "op": "attn", "B": B, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype,
            "window": window}


def sample(name, M, V, dtype):
    return {"name": name, "op": "sample", "M": M, "V": V, "dtype": dtype}


def plan(name, B, new, ctx, page, width):
    return {"name": name, "op": "plan", "B": B, "new": new, "ctx": ctx, "page": page, "width": width}


def append(name, T, hkv, d, page, blocks, dtype):
    return {"name": name, "op": "append", "T": T, "hkv": hkv, "d": d, "page": page, "blocks": blocks, "dtype": dtype}


def log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "sample", "sample", "plan", "append"])
    if op == "sample":
        M = log_uniform(rng, 1, 256)
        case = sample("", M, log_uniform(rng, 100, min(260000, 20000000 // M)), rng.choice(["f32", "bf16"]))
    elif op == "plan":
        case = plan("", log_uniform(rng, 1, 600), rng.choice(["1", "1-16", "first:%d,1-16" % log_uniform(rng, 17, 8192)]),
                    "0-%d" % log_uniform(rng, 10, 16000), rng.choice([8, 16, 48, 64]), 2048)
    elif op == "append":
        page = rng.choice([8, 16, 48, 64])
        case = append("", log_uniform(rng, 1, 8192), rng.choice([1, 2, 5, 8]), rng.choice([64, 128]), page, 131072 // page,
                      rng.choice(["bf16", "f16"]))
    else:
        hkv, group = rng.choice([(8, 4), (8, 8), (16, 1), (1, 16), (2, 7), (4, 6), (5, 3)])
        kind = rng.choice(["decode", "verify", "chunk", "mixed"])
        if kind == "decode":
            B, new, top = log_uniform(rng, 1, 64), "1", 100000
        elif kind == "verify":
            B, new, top = log_uniform(rng, 1, 48), "2-16", 16000
        elif kind == "chunk":
            B, new, top = rng.choice([1, 2]), "%d" % log_uniform(rng, 33, 4096), 8000
        else:
            B, new, top = rng.randint(2, 17), "first:%d,1-8" % log_uniform(rng, 17, 600), 4000
        top = min(top, 400000000 // (B * hkv * 128))  # the caches hold 2 GB at the most
        case = attn("", B, new, "0-%d" % log_uniform(rng, 10, top), hkv * group, hkv, rng.choice([64, 128]),
                    rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(["bf16", "f16"]), rng.choice([0, 0, 0, rng.randint(1, 4000)]))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def between(rs, text, n):
    lo, _, hi = text.partition("-")
    return rs.randint(int(lo), int(hi or lo) + 1, n).astype(np.int64)


def lengths(case, rs):
    """New and earlier tokens of each request; "first:N,..." gives the first request N new ones."""
    first, _, rest = case["new"].partition(",")
    new = between(rs, rest if first.startswith("first:") else case["new"], case["B"])
    if first.startswith("first:"):
        new[0] = int(first[6:])
    return new, between(rs, case["ctx"], case["B"])


def shapes(case):
    """Tokens and pages that a case of these lengths has at the most: the sizes of its buffers, whatever the seed."""
    first, _, rest = case["new"].partition(",")
    most = int((rest if first.startswith("first:") else case["new"]).partition("-")[2] or (rest or first).partition("-")[0])
    extra = int(first[6:]) if first.startswith("first:") else most
    ctx = case["ctx"].partition("-")
    top = int(ctx[2] or ctx[0])
    return {"tokens": extra + most * (case["B"] - 1), "longest": top + max(extra, most), "chunk": max(extra, most), "ctx": top}


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"attn": prepare_attn, "sample": prepare_sample, "plan": prepare_plan, "append": prepare_append}[case["op"]](case, rs, gen)


def prepare_attn(case, rs, gen):
    new, ctx = lengths(case, rs)
    size, page, seq = shapes(case), case["page"], ctx + new
    pages = -(-seq // page)
    width = -(-size["longest"] // page)
    n_blocks = int(pages.sum()) + 3
    # blocks handed out in the order of a server that has run for a while; what is not in use holds no block's number
    order = rs.permutation(n_blocks)
    table = np.full((case["B"], width), -1, np.int32)
    used = np.arange(width)[None, :] < pages[:, None]
    table[used] = order[: int(pages.sum())]
    dtype, tokens = TYPES[case["dtype"]], size["tokens"]
    kv = [torch.empty((n_blocks, page, case["hkv"], case["d"]), dtype=dtype, device="cuda").normal_(generator=gen) for _ in range(2)]
    q = torch.empty((tokens, case["hq"], case["d"]), dtype=dtype, device="cuda").normal_(generator=gen)
    return {"case": case, "q": q, "k": kv[0], "v": kv[1], "table": ints(table), "q_start": ints(np.concatenate([[0], np.cumsum(new)])),
            "seq": ints(seq), "longest": size["longest"], "chunk": size["chunk"], "out": torch.empty_like(q),
            "lse": torch.empty((tokens, case["hq"]), dtype=torch.float32, device="cuda")}


def prepare_sample(case, rs, gen):
    M, V = case["M"], case["V"]
    # a bulk of unlikely tokens and a few that the context makes likely
    logits = torch.empty((M, V), device="cuda").normal_(0.0, 2.0, generator=gen)
    likely = torch.randint(0, V, (M, 40), device="cuda", generator=gen)
    logits.scatter_add_(1, likely, torch.empty((M, 40), device="cuda").normal_(6.0, 2.5, generator=gen))
    logits[rs.randint(0, 4)::4, V // 2:V // 2 + V // 10] = -math.inf  # rows under a grammar
    pick = lambda values: torch.from_numpy(rs.choice(np.array(values), M)).cuda()  # noqa: E731
    return {"case": case, "logits": logits.to(TYPES[case["dtype"]]), "u": torch.rand(M, device="cuda", generator=gen),
            "temperature": pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3]).float(), "top_k": pick([0, 0, 1, 20, 50, 1000]).int(),
            "top_p": pick([1.0, 0.8, 0.9, 0.95, 0.99]).float(), "min_p": pick([0.0, 0.0, 0.02, 0.1]).float(),
            "tokens": torch.empty(M, dtype=torch.int32, device="cuda"), "probs": torch.empty(M, device="cuda")}


def prepare_plan(case, rs, gen):
    new, ctx = lengths(case, rs)
    size, page, B, width = shapes(case), case["page"], case["B"], case["width"]
    have = -(-ctx // page)
    total = int(have.sum()) + size["tokens"] // page + 2 * B
    order = rs.permutation(total)
    table = np.full((B, width), -1, np.int32)
    table[np.arange(width)[None, :] < have[:, None]] = order[: int(have.sum())]
    T = size["tokens"]
    one = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "ctx": ints(ctx), "new": ints(new), "table": ints(table), "free": ints(order[int(have.sum()):]),
            "q_start": one(B + 1), "seq": one(B), "slots": one(T), "positions": one(T), "taken": one(1)}


def prepare_append(case, rs, gen):
    T, hkv, d, dtype = case["T"], case["hkv"], case["d"], TYPES[case["dtype"]]
    # keys and values are slices of the fused projection's output, between queries of four times their heads
    fused = torch.empty((T, 6 * hkv, d), dtype=dtype, device="cuda").normal_(generator=gen)
    cache = [torch.zeros((case["blocks"], case["page"], hkv, d), dtype=dtype, device="cuda") for _ in range(2)]
    # the tokens' places run through pages that lie anywhere; the last few rows of a padded batch have none
    pages = -(-T // case["page"])
    slots = (rs.permutation(case["blocks"])[:pages, None] * case["page"] + np.arange(case["page"])[None, :]).reshape(-1)[:T]
    slots[T - T // 16:] = -1
    return {"case": case, "k_new": fused[:, 4 * hkv:5 * hkv], "v_new": fused[:, 5 * hkv:], "k": cache[0], "v": cache[1], "slots": ints(slots)}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": own_attn, "sample": own_sample, "plan": own_plan, "append": own_append}[op](state)
    return {"attn": plain_attn, "sample": plain_sample, "plan": plain_plan, "append": plain_append}[op](state)


def plain_attn(s):
    case = s["case"]
    B, hq, hkv, d, page = (case[n] for n in ("B", "hq", "hkv", "d", "page"))
    q_start, seq, longest, chunk = s["q_start"].long(), s["seq"].long(), s["longest"], s["chunk"]
    new = q_start[1:] - q_start[:-1]
    j = torch.arange(longest, device="cuda")
    block = s["table"].long()[:, j // page].clamp_min(0)
    held = (j < seq[:, None])[:, :, None, None]
    k = torch.where(held, s["k"][block, j % page].float(), 0.0)  # [B, longest, hkv, d]
    v = torch.where(held, s["v"][block, j % page].float(), 0.0)
    i = torch.arange(chunk, device="cuda")
    at = (q_start[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, chunk, hkv, hq // hkv, d)
    scores = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d), k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    scores = scores.view(B, hkv, hq // hkv, chunk, longest)
    p = (seq - new)[:, None] + i
    seen = (j <= p[:, :, None]) & (j < seq[:, None, None])
    if case["window"]:
        seen &= j > p[:, :, None] - case["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores.view(B, hkv, -1, longest), v.permute(0, 2, 1, 3)).view(B, hkv, hq // hkv, chunk, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0]
    # back to rows of tokens; rows past the last request's are padding and stay empty
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(q_start[1:], t, right=True)
    real = b < B
    b = b.clamp_max(B - 1)
    i = torch.where(real, t - q_start[b], 0)
    out = torch.where(real[:, None, None], o.permute(0, 3, 1, 2, 4).reshape(B, chunk, hq, d)[b, i], 0.0)
    lse = torch.where(real[:, None], lse.permute(0, 3, 1, 2).reshape(B, chunk, hq)[b, i], -math.inf)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def plain_sample(s):
    logits = s["logits"].double()
    M, V = logits.shape
    logits = torch.where(logits.isnan(), -math.inf, logits)
    temperature, top_k, top_p, min_p = (s[n].double()[:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    ordered, index = torch.sort(logits, dim=1, descending=True, stable=True)
    greedy = temperature <= 0
    w = torch.exp((ordered - ordered[:, :1]) / torch.where(greedy, 1.0, temperature))
    rank = torch.arange(V, device="cuda")[None, :]
    first = (rank < top_k) | (top_k <= 0)
    w_k = torch.where(first, w, 0.0)
    sums = w_k.cumsum(1)
    kept = first & ((sums - w_k < top_p * sums[:, -1:]) | (top_p >= 1) | (rank == 0)) & (w >= min_p)
    kept = torch.where(greedy, rank == 0, kept)
    mass = torch.zeros_like(w).scatter_(1, index, torch.where(kept, w, 0.0))
    cdf = mass.cumsum(1)
    token = (cdf <= s["u"].double()[:, None] * cdf[:, -1:]).sum(1, keepdim=True).clamp_max(V - 1)
    return {"tokens": token[:, 0].int(), "probs": (mass.gather(1, token) / cdf[:, -1:])[:, 0].float()}


def plain_plan(s):
    case = s["case"]
    page, width, B = case["page"], case["width"], case["B"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    seq = ctx + new
    q_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    have, need = (ctx + page - 1) // page, (seq + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have)
    col = torch.arange(width, device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    table.copy_(torch.where(fresh, free[(first[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)], table))
    t = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(q_start[1:], t, right=True)
    real = b < B
    b = b.clamp_max(B - 1)
    position = torch.where(real, ctx[b] + t - q_start[b], -1)
    slot = torch.where(real, table[b, position.clamp_min(0) // page].long() * page + position % page, -1)
    return {"q_start": q_start.int(), "seq": seq.int(), "slots": slot.int(), "positions": position.int(), "table": table,
            "taken": (need - have).sum().int().view(1)}


def plain_append(s):
    slots = s["slots"].long()
    real = (slots >= 0)[:, None, None]
    page = s["case"]["page"]
    at = slots.clamp_min(0)
    for new, cache in ((s["k_new"], s["k"]), (s["v_new"], s["v"])):
        # a padding row is written over the first row of its batch again
        src = torch.where(real, new, new[:1])
        at = torch.where(real[:, 0, 0], slots, slots[0])
        cache[at // page, at % page] = src
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ the library's calls
def handles(s):
    """What a program keeps next to its buffers: the cache's description and a workspace."""
    if "ws" not in s:
        from moe_decode_gb300 import api
        s["api"] = api
        if "k" in s:
            s["cache"] = api.KvCache(s["k"], s["v"])
        s["ws"] = api.paged_workspace(s["q"].shape[1], s["cache"]) if "q" in s else api.paged_workspace()
    return s["api"]


def own_attn(s):
    handles(s).paged_attention(s["q"], s["cache"], s["table"], s["q_start"], s["seq"], s["out"], s["ws"], lse=s["lse"],
                               window=s["case"]["window"])
    return {"out": s["out"], "lse": s["lse"]}


def own_sample(s):
    handles(s).sample(s["logits"], s["u"], s["tokens"], probs=s["probs"], temperature=s["temperature"], top_k=s["top_k"],
                      top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": s["tokens"], "probs": s["probs"]}


def own_plan(s):
    handles(s).paged_plan(s["ctx"], s["new"], s["free"], s["table"], s["case"]["page"], s["q_start"], s["seq"], s["slots"],
                          s["taken"], s["ws"], positions=s["positions"])
    return {"q_start": s["q_start"], "seq": s["seq"], "slots": s["slots"], "positions": s["positions"], "table": s["table"],
            "taken": s["taken"]}


def own_append(s):
    handles(s).paged_append(s["k_new"], s["v_new"], s["slots"], s["cache"], s["ws"])
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ what a pass cannot do without
def mean_of(text):
    lo, _, hi = text.partition("-")
    return (int(lo) + int(hi or lo)) / 2


def work(case):
    if case["op"] == "sample":
        n = case["M"] * case["V"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["M"] * 28, "flops": 6 * n}
    if case["op"] == "append":
        real = case["T"] - case["T"] // 16
        return {"bytes": 4 * real * case["hkv"] * case["d"] * 2 + 4 * case["T"], "flops": 0}
    first, _, rest = case["new"].partition(",")
    new = [mean_of(rest if rest else first)] * case["B"]
    if first.startswith("first:"):
        new[0] = float(first[6:])
    ctx, T = mean_of(case["ctx"]), shapes(case)["tokens"]
    if case["op"] == "plan":
        fresh = sum(n / case["page"] for n in new)
        return {"bytes": int(4 * (5 * case["B"] + 2 * T + 2 * fresh)), "flops": 8 * T}
    pairs, keys = 0.0, 0.0
    for n in new:
        w = case["window"] or n + ctx + 1
        mean = min(w, ctx + n / 2)
        pairs += n * mean
        keys += min(ctx + n, w + n)
    tokens = sum(new)
    size = 2 * (2 * keys * case["hkv"] * case["d"] + 2 * tokens * case["hq"] * case["d"]) + 4 * tokens * case["hq"]
    return {"bytes": int(size), "flops": int(4 * pairs * case["hq"] * case["d"])}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    return {"attn": exact_attn, "sample": exact_sample, "append": exact_append}[case["op"]](prepare(case, seed))


def exact_attn(s):
    case = s["case"]
    T, hq, d = s["q"].shape
    group, page = hq // case["hkv"], case["page"]
    out = torch.zeros((T, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    q_start, seq, table = s["q_start"].tolist(), s["seq"].tolist(), s["table"].cpu().numpy()
    for b in range(case["B"]):
        lo, hi, n = q_start[b], q_start[b + 1], seq[b]
        where = torch.from_numpy(np.repeat(table[b].astype(np.int64) * page, page)[:n] + np.arange(n) % page).cuda()
        for g in range(case["hkv"]):
            k = s["k"][:, :, g].reshape(-1, d)[where].double()
            v = s["v"][:, :, g].reshape(-1, d)[where].double()
            # a few thousand rows at a time
            for a in range(lo, hi, 2048):
                z = min(hi, a + 2048)
                q = s["q"][a:z, g * group:(g + 1) * group].double()
                place = torch.arange(n - hi + a, n - hi + z, device="cuda")
                first = (place - case["window"] + 1).clamp_min(0) if case["window"] else torch.zeros_like(place)
                key = torch.arange(n, device="cuda")
                hidden = (key[None, :] > place[:, None]) | (key[None, :] < first[:, None])
                dots = torch.einsum("tgd,kd->gtk", q, k) / math.sqrt(d)
                dots[:, hidden] = -math.inf
                z_lse = torch.logsumexp(dots, -1)
                out[a:z, g * group:(g + 1) * group] = torch.einsum("gtk,kd->tgd", torch.exp(dots - z_lse[..., None]), v)
                lse[a:z, g * group:(g + 1) * group] = z_lse.T
    return {"out": out, "lse": lse}


def exact_sample(s):
    logits = s["logits"].double().cpu().numpy()
    u, temperature, top_p, min_p = (s[n].cpu().numpy().astype(np.float64) for n in ("u", "temperature", "top_p", "min_p"))
    top_k = s["top_k"].cpu().numpy()
    probs = np.zeros(len(u))
    for r, row in enumerate(logits):
        if temperature[r] <= 0:
            probs[r] = 1.0
            continue
        order = np.argsort(-row, kind="stable")
        if top_k[r] > 0:
            order = order[: top_k[r]]
        p = np.exp((row[order] - row[order[0]]) / temperature[r])
        keep = len(order)
        if top_p[r] < 1:
            keep = max(1, min(keep, int(np.searchsorted(np.cumsum(p), top_p[r] * p.sum(), side="left")) + 1))
        keep = min(keep, int((p >= min_p[r]).sum()))
        chosen = np.sort(order[:keep])
        p = np.exp((row[chosen] - row[order[0]]) / temperature[r])
        c = np.cumsum(p)
        at = min(int(np.searchsorted(c, u[r] * c[-1], side="right")), keep - 1)
        probs[r] = p[at] / c[-1]
    return {"tokens": None, "probs": torch.from_numpy(probs)}


def exact_append(s):
    page, slots = s["case"]["page"], s["slots"].cpu().numpy()
    got = {}
    for name in ("k", "v"):
        rows = s[name].double().reshape(-1, *s[name].shape[2:])
        at = torch.from_numpy(np.nonzero(slots >= 0)[0]).cuda()
        rows.index_copy_(0, s["slots"].long()[at], s[name + "_new"][at].double())
        got[name] = rows.view(-1, page, *rows.shape[1:])
    return got
