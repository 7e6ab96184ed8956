"""More operators of the paged step, as they are measured: rotary positions, alone and in one pass with the write of new keys and values
into the cache; the write into and the reading back of a cache of 8-bit values; the attention of new tokens over such a cache; and the
verification of a tree of drafted tokens (its masks and positions, and its attention over the cache).

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes one pass (the plain form in
elementary torch operations, or the library's calls where ``own`` is true), ``exact`` gives the same outputs from the definitions in
64 bits.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
PLAIN = {"rd": 128, "pairs": "half", "base": 10000.0, "scaling": "none", "factor": 1.0, "context": 0}


# ------------------------------------------------------------------ cases
def listed():
    far = {"rd": 128, "pairs": "half", "base": 1000000.0, "scaling": "yarn", "factor": 4.0, "context": 32768}
    part = {"rd": 64, "pairs": "interleaved", "base": 10000.0, "scaling": "none", "factor": 1.0, "context": 0}
    return [
        # queries and keys of 32 streams that each decode a token, far into contexts longer than the model was made for: latency
        rope("rope_decode", 32, 32, 8, 128, "bf16", 131000, far),
        # those of a full chunk, neighbouring pairs in half of the head
        rope("rope_chunk", 8192, 32, 8, 128, "f16", 30000, part),
        # a verify step's keys and values rotated, quantised and written, its queries rotated
        append("append8_verify", 96, 32, 8, 128, 16, 2048, "bf16", "e4m3", 16000, PLAIN),
        # the same of a full chunk
        append("append8_chunk", 8192, 32, 8, 128, 16, 8192, "bf16", "e4m3", 30000, far),
        # the keys and values of an accepted path read back, to be moved
        read("read8_path", 48, 8, 128, 16, 4096, "bf16"),
        # a long context read back for the chunk of a prompt that attends over it
        read("read8_context", 65521, 8, 128, 64, 2048, "bf16"),
        # one stream, one new token, a short history, over the cache of 8-bit values
        attn("attn8_decode_short", 1, "1", "1000", 32, 8, 128, 16, "bf16", "e4m3", 0),
        # 32 streams verifying chains of 6 speculated tokens, histories of all lengths
        attn("attn8_verify_batch", 32, "6", "300-16000", 32, 8, 128, 16, "bf16", "e4m3", 0),
        # a few streams deep into long documents, one token each: the cache's bandwidth
        attn("attn8_decode_long", 4, "1", "120001-131070", 64, 8, 128, 64, "f16", "e4m3", 0),
        # one stream that verifies a tree of 16 drafted tokens
        tree("tree_one", 1, "16", "1500", 32, 8, 128, 16, "bf16", "bf16"),
        # many streams with trees of up to 64
        tree("tree_batch", 24, "33-64", "200-12000", 32, 8, 128, 16, "bf16", "bf16"),
        # small trees over the cache of 8-bit values
        tree("tree8_batch", 16, "4-21", "200-12000", 32, 8, 128, 32, "bf16", "e4m3"),
    ]


def rope(name, T, hq, hkv, d, dtype, top, angles):
    return {"name": name, "op": "rope", "T": T, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "top": top, **angles}


def append(name, T, hq, hkv, d, page, blocks, dtype, cache, top, angles):
    return {"name": name, "op": "append", "T": T, "hq": hq, "hkv": hkv, "d": d, "page": page, "blocks": blocks, "dtype": dtype, "cache": cache,
            "top": top, **angles}


def read(name, T, hkv, d, page, blocks, dtype):
    return {"name": name, "op": "read", "T": T, "hkv": hkv, "d": d, "page": page, "blocks": blocks, "dtype": dtype}


def attn(name, B, new, ctx, hq, hkv, d, page, dtype, cache, window):
    return {"name": name, "op": "attn", "B": B, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype, "cache": cache,
            "window": window}


def tree(name, B, new, ctx, hq, hkv, d, page, dtype, cache):
    return {**attn(name, B, new, ctx, hq, hkv, d, page, dtype, cache, 0), "op": "tree"}


def log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw_angles(rng, d):
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn", "bands"])
    return {"rd": rng.choice([d, d, d // 2, d // 4]), "pairs": rng.choice(["half", "interleaved"]), "base": rng.choice([10000.0, 500000.0]),
            "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]), "context": 0 if scaling == "none" else 8192}


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn", "tree", "tree"])
    hkv, group = rng.choice([(8, 4), (8, 8), (16, 1), (1, 16), (2, 7), (4, 6), (5, 3)])
    d, page, dtype = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "f16"])
    if op == "rope":
        d = rng.choice([64, 128, 128, 192])
        case = rope("", log_uniform(rng, 1, 4096), hkv * group, hkv, d, dtype, log_uniform(rng, 100, 1000000), draw_angles(rng, d))
    elif op == "append":
        case = append("", log_uniform(rng, 1, 8192), hkv * min(group, 4), hkv, d, page, 131072 // page, dtype, rng.choice(["e4m3", "e4m3", dtype]),
                      log_uniform(rng, 100, 1000000), draw_angles(rng, d))
    elif op == "read":
        case = read("", log_uniform(rng, 1, 65000), min(hkv, 8), d, page, 131072 // page, dtype)
    elif op == "attn":
        kind = rng.choice(["decode", "verify", "chunk"])
        if kind == "decode":
            B, new, top = log_uniform(rng, 1, 64), "1", 100000
        elif kind == "verify":
            B, new, top = log_uniform(rng, 1, 48), "2-16", 16000
        else:
            B, new, top = rng.randint(1, 9), "first:%d,1-8" % log_uniform(rng, 17, 600), 4000
        top = min(top, 400000000 // (B * hkv * 128))
        case = attn("", B, new, "0-%d" % log_uniform(rng, 10, top), hkv * group, hkv, d, page, dtype, "e4m3", rng.choice([0, 0, rng.randint(1, 4000)]))
    else:
        B = log_uniform(rng, 1, 24)
        case = tree("", B, "1-%d" % rng.randint(2, 64), "0-%d" % log_uniform(rng, 10, min(12000, 200000000 // (B * hkv * 128))), hkv * group, hkv, d,
                    page, dtype, rng.choice(["e4m3", dtype]))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


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
    return {"tokens": extra + most * (case["B"] - 1), "longest": int(ctx[2] or ctx[0]) + max(extra, most), "chunk": max(extra, most)}


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def frequencies(case):
    """Radians a position for each pair, in 64 bits, and the factor of the rotated values."""
    rd, base, c, L = case["rd"], case["base"], case["factor"], case["context"]
    if case["scaling"] == "ntk":
        base *= c ** (rd / (rd - 2))
    f = base ** (-np.arange(0, rd, 2) / rd)
    if case["scaling"] == "linear":
        f = f / c
    if case["scaling"] == "yarn":  # pairs that turn more than 32 times in the first context stay, those of less than one turn are stretched
        at = [rd * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        kept = 1 - np.clip((np.arange(rd // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f / c * (1 - kept) + f * kept, 0.1 * math.log(c) + 1
    if case["scaling"] == "bands":  # wavelengths up to a quarter of the first context stay, those beyond it are stretched
        kept = np.clip((L * f / (2 * math.pi) - 1) / (4 - 1), 0, 1)
        return f / c * (1 - kept) + f * kept, 1.0
    return f, 1.0


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"rope": prepare_rope, "append": prepare_append, "read": prepare_read, "attn": prepare_attn, "tree": prepare_attn}
    return make[case["op"]](case, rs, gen)


def normal(gen, dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def prepare_rope(case, rs, gen):
    T, hq, hkv, d, dtype = case["T"], case["hq"], case["hkv"], case["d"], TYPES[case["dtype"]]
    freqs, scale = frequencies(case)
    fused = normal(gen, dtype, T, hq + 2 * hkv, d)  # the fused projection's output
    at = rs.randint(0, case["top"], T)
    at[T - T // 16:] = -1  # the last few rows of a padded batch
    return {"case": case, "q": fused[:, :hq], "k": fused[:, hq:hq + hkv], "v": fused[:, hq + hkv:], "positions": ints(at),
            "freqs": torch.from_numpy(freqs).cuda(), "scale": scale,
            "q_out": torch.zeros((T, hq, d), dtype=dtype, device="cuda"), "k_out": torch.zeros((T, hkv, d), dtype=dtype, device="cuda")}


def empty_cache(case, blocks):
    """K and V, and where they are codes the exponents of their scales: one byte for each token and head."""
    shape = (blocks, case["page"], case["hkv"], case["d"])
    if case.get("cache", "e4m3") != "e4m3":
        return {n: torch.zeros(shape, dtype=TYPES[case["cache"]], device="cuda") for n in ("k", "v")}
    s = {n: torch.zeros(shape, dtype=torch.uint8, device="cuda") for n in ("k", "v")}
    return {**s, **{n + "_scale": torch.zeros((blocks, case["hkv"], case["page"]), dtype=torch.uint8, device="cuda") for n in ("k", "v")}}


def places(case, rs, T):
    """Slots of T tokens: they run through pages that lie anywhere."""
    pages = -(-T // case["page"])
    return (rs.permutation(case["blocks"])[:pages, None] * case["page"] + np.arange(case["page"])[None, :]).reshape(-1)[:T]


def prepare_append(case, rs, gen):
    s = prepare_rope(case, rs, gen)
    slots = places(case, rs, case["T"])
    slots[case["T"] - case["T"] // 16:] = -1
    kv = {"cache_" + n: t for n, t in empty_cache(case, case["blocks"]).items()}
    return {**s, **kv, "slots": ints(slots)}


def filled_cache(case, blocks, gen):
    cache = empty_cache(case, blocks)
    for n in ("k", "v"):
        # tokens of different sizes, some pages at a time
        for at in range(0, blocks, 4096):
            x = normal(gen, torch.float32, *cache[n][at:at + 4096].shape)
            x *= torch.exp(normal(gen, torch.float32, *x.shape[:3], 1) * (0.1 if n == "k" else 0.7))
            if "k_scale" in cache:
                codes, e = quantised(x.to(TYPES[case["dtype"]]))
                cache[n][at:at + 4096] = codes.view(torch.uint8)
                cache[n + "_scale"][at:at + 4096] = e.transpose(1, 2)
            else:
                cache[n][at:at + 4096] = x.to(cache[n].dtype)
    return cache


def prepare_read(case, rs, gen):
    cache = filled_cache(case, case["blocks"], gen)
    T = case["T"]
    slots = places(case, rs, T)
    if T < 1000:  # single tokens out of their pages
        slots = rs.permutation(case["blocks"] * case["page"])[:T]
    slots[T - T // 16:] = -1
    out = [torch.zeros((T, case["hkv"], case["d"]), dtype=TYPES[case["dtype"]], device="cuda") for _ in range(2)]
    return {"case": case, **cache, "slots": ints(slots), "k_out": out[0], "v_out": out[1]}


def prepare_attn(case, rs, gen):
    new, ctx = lengths(case, rs)
    size, page, seq = shapes(case), case["page"], ctx + new
    pages = -(-seq // page)
    width = -(-size["longest"] // page)
    n_blocks = int(pages.sum()) + 3
    # blocks handed out in the order of a server that has run for a while; what is not in use holds no block's number
    order = rs.permutation(n_blocks)
    table = np.full((case["B"], width), -1, np.int32)
    table[np.arange(width)[None, :] < pages[:, None]] = order[: int(pages.sum())]
    dtype, T = TYPES[case["dtype"]], size["tokens"]
    # drafted tokens hang from one of the few before them, or from the context's last
    start = np.concatenate([[0], np.cumsum(new)])
    parents = np.full(T, -1)
    for b in range(case["B"]):
        i = np.arange(new[b])
        parents[start[b]:start[b + 1]] = np.where(rs.rand(new[b]) < 0.1, -1, i - 1 - np.minimum(rs.geometric(0.35, new[b]) - 1, i))
    return {"case": case, "q": normal(gen, dtype, T, case["hq"], case["d"]), **filled_cache(case, n_blocks, gen), "table": ints(table),
            "q_start": ints(start), "seq": ints(seq), "longest": size["longest"], "chunk": size["chunk"], "parents": ints(parents),
            "masks": torch.zeros(T, dtype=torch.int64, device="cuda"), "positions": torch.zeros(T, dtype=torch.int32, device="cuda"),
            "out": torch.zeros((T, case["hq"], case["d"]), dtype=dtype, device="cuda"),
            "lse": torch.zeros((T, case["hq"]), dtype=torch.float32, device="cuda")}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": own_rope, "append": own_append, "read": own_read, "attn": own_attn, "tree": own_tree}[op](state)
    return {"rope": plain_rope, "append": plain_append, "read": plain_read, "attn": plain_attn, "tree": plain_tree}[op](state)


def power(e):
    """2^e for whole e in -126 .. 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def quantised(x):
    """Codes of each row of the last dimension, and the byte that holds the exponent of its scale: the least one that keeps them in range."""
    m, e = torch.frexp(x.float().abs().amax(-1, keepdim=True))
    e = torch.where(m > 0, (e - 9 + (m > 0.875).int()).clamp_min(-127), -127)
    return (x.float() * power(-e)).to(E4M3), (e + 127).to(torch.uint8)[..., 0]


def rotated(x, s):
    case = s["case"]
    rd = case["rd"]
    angle = s["positions"].double()[:, None] * s["freqs"]
    c, n = ((f(angle) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.float()
    half = case["pairs"] == "half"
    first, second = (y[..., : rd // 2], y[..., rd // 2:rd]) if half else (y[..., 0:rd:2], y[..., 1:rd:2])
    a, b = first * c - second * n, first * n + second * c
    turned = torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, y[..., rd:]], -1).to(x.dtype)


def plain_rope(s):
    real = (s["positions"] >= 0)[:, None, None]
    return {n: torch.where(real, rotated(s[n], s), s[n + "_out"]) for n in ("q", "k")}


def plain_append(s):
    case, slots = s["case"], s["slots"].long()
    real = (slots >= 0)[:, None, None]
    got = {"q": torch.where(real, rotated(s["q"], s), s["q_out"])}
    # a padding row is written over the first row of its batch again
    at = torch.where(slots >= 0, slots, slots[:1])
    block, token = at // case["page"], at % case["page"]
    for n, x in (("k", rotated(s["k"], s)), ("v", s["v"])):
        x = torch.where(real, x, x[:1])
        if case["cache"] == "e4m3":
            codes, e = quantised(x)
            s["cache_" + n][block, token] = codes.view(torch.uint8)
            s["cache_" + n + "_scale"].transpose(1, 2)[block, token] = e
            got[n], got[n + "_scale"] = s["cache_" + n].view(E4M3), s["cache_" + n + "_scale"]
        else:
            s["cache_" + n][block, token] = x
            got[n] = s["cache_" + n]
    return got


def values(s, n, block, token):
    """Keys or values [..., heads, d] in fp32 of the cache's places."""
    if n + "_scale" not in s:
        return s[n][block, token].float()
    return s[n][block, token].view(E4M3).float() * power(s[n + "_scale"].transpose(1, 2)[block, token].int() - 127)[..., None]


def plain_read(s):
    page, slots = s["case"]["page"], s["slots"].long()
    at = slots.clamp_min(0)
    real = (slots >= 0)[:, None, None]
    return {n: torch.where(real, values(s, n, at // page, at % page).to(s["k_out"].dtype), s[n + "_out"]) for n in ("k", "v")}


def plain_attn(s, seen_new=None):
    case = s["case"]
    B, hq, hkv, d, page = (case[n] for n in ("B", "hq", "hkv", "d", "page"))
    q_start, seq, longest, chunk = s["q_start"].long(), s["seq"].long(), s["longest"], s["chunk"]
    new = q_start[1:] - q_start[:-1]
    j = torch.arange(longest, device="cuda")
    block = s["table"].long()[:, j // page].clamp_min(0)
    held = (j < seq[:, None])[:, :, None, None]
    k = torch.where(held, values(s, "k", block, j % page), 0.0)  # [B, longest, hkv, d]
    v = torch.where(held, values(s, "v", block, j % page), 0.0)
    i = torch.arange(chunk, device="cuda")
    at = (q_start[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, chunk, hkv, hq // hkv, d)
    scores = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d), k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    scores = scores.view(B, hkv, hq // hkv, chunk, longest)
    p = (seq - new)[:, None] + i
    seen = (j <= p[:, :, None]) & (j < seq[:, None, None])
    if case["window"]:
        seen &= j > p[:, :, None] - case["window"]
    if seen_new is not None:  # of the request's own new tokens those that the mask names
        place = (j - (seq - new)[:, None])[:, None, :].expand(B, chunk, longest)
        seen &= (place < 0) | torch.gather(seen_new[:, :chunk], 2, place.clamp(0, 63))
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


def plain_tree(s):
    B, T = s["case"]["B"], s["q"].shape[0]
    q_start, seq = s["q_start"].long(), s["seq"].long()
    new = q_start[1:] - q_start[:-1]
    i = torch.arange(64, device="cuda")
    row = (q_start[:-1, None] + i).clamp_max(T - 1)
    parent = torch.where(i < new[:, None], s["parents"].long()[row], -1)
    up = (parent[:, :, None] == i).float() + torch.eye(64, device="cuda")  # a token, and the one it hangs from
    up = torch.matmul(up, up).clamp_max(1.0)  # up to 2 steps
    up = torch.matmul(up, up).clamp_max(1.0)
    up = torch.matmul(up, up).clamp_max(1.0)
    up = torch.matmul(up, up).clamp_max(1.0)
    up = torch.matmul(up, up).clamp_max(1.0)
    up = torch.matmul(up, up) > 0  # up to 64
    masks = (up.long() << i).sum(-1)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(q_start[1:], t, right=True)
    real = b < B
    b = b.clamp_max(B - 1)
    at = torch.where(real, t - q_start[b], 0)
    depth = up.sum(-1)[b, at] - 1
    return {**plain_attn(s, up), "masks": torch.where(real, masks[b, at], 0),
            "positions": torch.where(real, (seq - new)[b] + depth, -1).int()}


# ------------------------------------------------------------------ the library's calls
def handles(s):
    """What a program keeps next to its buffers: the angles, the cache's description and a workspace."""
    if "api" not in s:
        from moe_decode_gb300 import api
        case = s["case"]
        s["api"] = api
        if "freqs" in s:
            s["angles"] = api.Rope(case["rd"], base=case["base"], interleaved=case["pairs"] == "interleaved", scaling=case["scaling"],
                                   factor=case["factor"], context=case["context"])
        prefix = "cache_" if "cache_k" in s else ""
        if prefix + "k_scale" in s:
            s["handle"] = api.KvCache8(*(s[prefix + n] for n in ("k", "v", "k_scale", "v_scale")))
        elif case["op"] != "rope":
            s["handle"] = api.KvCache(s[prefix + "k"], s[prefix + "v"])
        s["ws"] = api.paged_workspace(case["hq"], s["handle"]) if "table" in s else api.paged_workspace()
    return s["api"]


def own_rope(s):
    handles(s).rope(s["q"], s["k"], s["positions"], s["angles"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def own_append(s):
    handles(s).paged_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["angles"], s["handle"], s["ws"], q_out=s["q_out"])
    got = {"q": s["q_out"]}
    for n in ("k", "v"):
        if "cache_k_scale" in s:
            got[n], got[n + "_scale"] = s["cache_" + n].view(E4M3), s["cache_" + n + "_scale"]
        else:
            got[n] = s["cache_" + n]
    return got


def own_read(s):
    handles(s).paged_read(s["handle"], s["slots"], s["k_out"], s["v_out"], s["ws"])
    return {"k": s["k_out"], "v": s["v_out"]}


def own_attn(s):
    handles(s).paged_attention(s["q"], s["handle"], s["table"], s["q_start"], s["seq"], s["out"], s["ws"], lse=s["lse"],
                               window=s["case"]["window"])
    return {"out": s["out"], "lse": s["lse"]}


def own_tree(s):
    api = handles(s)
    api.tree_plan(s["parents"], s["q_start"], s["seq"], s["masks"], s["positions"], s["ws"])
    api.paged_attention(s["q"], s["handle"], s["table"], s["q_start"], s["seq"], s["out"], s["ws"], lse=s["lse"], tree_masks=s["masks"])
    return {"out": s["out"], "lse": s["lse"], "masks": s["masks"], "positions": s["positions"]}


# ------------------------------------------------------------------ what a pass cannot do without
def mean_of(text):
    lo, _, hi = text.partition("-")
    return (int(lo) + int(hi or lo)) / 2


def work(case):
    op = case["op"]
    if op in ("rope", "append"):
        real = case["T"] - case["T"] // 16
        q, kv = 2 * case["hq"] * case["d"], case["hkv"] * case["d"]
        held = case["hkv"] * (case["d"] + 1) if case.get("cache") == "e4m3" else 2 * kv
        size = real * (2 * q + 4 * kv) if op == "rope" else real * (2 * q + 4 * kv + 2 * held) + 4 * case["T"]
        return {"bytes": size + 4 * case["T"] + 4 * case["rd"], "flops": 3 * real * (case["hq"] + case["hkv"]) * case["rd"]}
    if op == "read":
        real = case["T"] - case["T"] // 16
        return {"bytes": 2 * real * case["hkv"] * (3 * case["d"] + 1) + 4 * case["T"], "flops": 0}
    first, _, rest = case["new"].partition(",")
    new = [mean_of(rest if rest else first)] * case["B"]
    if first.startswith("first:"):
        new[0] = float(first[6:])
    ctx = mean_of(case["ctx"])
    pairs, keys = 0.0, 0.0
    for n in new:
        w = case["window"] or n + ctx + 1
        pairs += n * min(w, ctx + n / 2)
        keys += min(ctx + n, w + n)
    tokens = sum(new)
    held = case["d"] + 1 if case["cache"] == "e4m3" else 2 * case["d"]
    size = 2 * keys * case["hkv"] * held + 4 * tokens * case["hq"] * case["d"] + 4 * tokens * case["hq"] + (16 * tokens if op == "tree" else 0)
    return {"bytes": int(size), "flops": int(4 * pairs * case["hq"] * case["d"])}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {n: kept(turned(s[n], s), s["positions"], s[n + "_out"]) for n in ("q", "k")}
    return {"append": exact_append, "read": exact_read, "attn": exact_attn, "tree": exact_attn}[case["op"]](s)


def kept(x, places, before):
    return torch.where(places[:, None, None] < 0, before.double(), x)


def turned(x, s):
    """Each pair as a complex number times e^(i angle)."""
    case, x = s["case"], x.double()
    rd = case["rd"]
    angle = torch.outer(s["positions"].double(), s["freqs"])[:, None, :]
    by = torch.polar(torch.full_like(angle, s["scale"]), angle)
    order = torch.arange(rd, device="cuda").view(2, -1).T if case["pairs"] == "half" else torch.arange(rd, device="cuda").view(-1, 2)
    z = torch.view_as_complex(x[..., order].contiguous()) * by
    y = x.clone()
    y[..., order] = torch.view_as_real(z)
    return y


def exact_append(s):
    case, slots = s["case"], s["slots"].long()
    at = torch.nonzero(slots >= 0)[:, 0]
    got = {"q": kept(turned(s["q"], s), s["slots"], s["q_out"])}
    for n in ("k", "v"):
        cache = s["cache_" + n]
        if case["cache"] == "e4m3":
            # a rotated key's code goes by which side of a border it comes to lie on: that has no 64-bit value; the scale is a whole number
            if n == "v":
                rows = cache.view(E4M3).double().view(-1, *cache.shape[2:])
                rows[slots[at]] = nearest_code(s["v"][at])
                got[n] = rows.view(cache.shape)
            else:
                got[n] = None
            got[n + "_scale"] = None
            continue
        rows = cache.double().view(-1, *cache.shape[2:])
        rows[slots[at]] = (turned(s["k"], s) if n == "k" else s["v"].double())[at]
        got[n] = rows.view(cache.shape)
    return got


def nearest_code(x):
    """The e4m3 number nearest to x over its row's scale, an even code where two are as near."""
    table = np.array([(m + 8 * (e > 0)) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127])
    table = torch.from_numpy(table).cuda()
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448)).clamp_min(-127)
    y = x.abs() / torch.pow(2.0, e)
    above = torch.searchsorted(table, y.contiguous()).clamp(1, 126)
    lo, hi = table[above - 1], table[above]
    up = (hi - y < y - lo) | ((hi - y == y - lo) & (above % 2 == 0))
    return torch.where(up, hi, lo) * torch.sign(x)


def held(s, n):
    """All of the cache's keys or values in 64 bits, one row a slot."""
    x = s[n].view(E4M3).double() if n + "_scale" in s else s[n].double()
    if n + "_scale" in s:
        x *= torch.pow(2.0, s[n + "_scale"].double() - 127).transpose(1, 2)[..., None]
    return x.reshape(-1, *x.shape[2:])


def exact_read(s):
    return {n: kept(held(s, n)[s["slots"].long().clamp_min(0)], s["slots"], s[n + "_out"]) for n in ("k", "v")}


def exact_attn(s):
    case = s["case"]
    T, hq, d = s["q"].shape
    group, page = hq // case["hkv"], case["page"]
    out = torch.zeros((T, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    q_start, seq, table, parents = s["q_start"].tolist(), s["seq"].tolist(), s["table"].cpu().numpy(), s["parents"].tolist()
    for b in range(case["B"]):
        lo, hi, n = q_start[b], q_start[b + 1], seq[b]
        where = torch.from_numpy(np.repeat(table[b].astype(np.int64) * page, page)[:n] + np.arange(n) % page).cuda()
        block, token = where // page, where % page
        place = torch.arange(n - hi + lo, n, device="cuda")
        key = torch.arange(n, device="cuda")
        first = (place - case["window"] + 1).clamp_min(0) if case["window"] else torch.zeros_like(place)
        hidden = (key[None, :] > place[:, None]) | (key[None, :] < first[:, None])
        if case["op"] == "tree":
            on_path = np.zeros((hi - lo, hi - lo), bool)
            for i in range(hi - lo):
                j = i
                while j >= 0:
                    on_path[i, j] = True
                    j = parents[lo + j]
            hidden[:, n - hi + lo:] |= torch.from_numpy(~on_path).cuda()
        for g in range(case["hkv"]):
            k, v = (s[x][block, token, g] for x in ("k", "v"))
            if "k_scale" in s:
                k, v = (y.view(E4M3).double() * torch.pow(2.0, s[x + "_scale"][block, g, token].double() - 127)[:, None]
                        for x, y in (("k", k), ("v", v)))
            q = s["q"][lo:hi, g * group:(g + 1) * group].double()
            dots = torch.einsum("tgd,kd->gtk", q, k.double()) / math.sqrt(d)
            dots[:, hidden] = -math.inf
            z = torch.logsumexp(dots, -1)
            out[lo:hi, g * group:(g + 1) * group] = torch.einsum("gtk,kd->tgd", torch.exp(dots - z[..., None]), v.double())
            lse[lo:hi, g * group:(g + 1) * group] = z.T
    return {"out": out, "lse": lse, **({"masks": None, "positions": None} if case["op"] == "tree" else {})}
