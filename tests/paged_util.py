"""Plain references of the paged step's operators, in 64 bits, and inputs for
their tests."""
import math

import numpy as np
import torch


def make_cache(n_blocks, page, heads, d, dtype, seed, layout="bthd"):
    """(K, V) [n_blocks, page, heads, d] views of the layout's own buffers."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def one(*shape):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)

    if layout == "bthd":
        return one(n_blocks, page, heads, d), one(n_blocks, page, heads, d)
    if layout == "bhtd":
        return tuple(one(n_blocks, heads, page, d).transpose(1, 2) for _ in range(2))
    both = one(n_blocks, 2, page, heads, d)  # K and V of a block side by side
    return both[:, 0], both[:, 1]


def make_step(lens, page, heads, kv_heads, d, dtype, seed, layout="bthd", window=0, pad=0, width=None, poison=True):
    """Inputs of paged_attention for requests lens = [(seq, new), ...]. Blocks
    lie in a shuffled order; whatever no row may read is poisoned: the rest of
    each request's last page with NaN, table entries that hold no visible key
    with -1."""
    rs = np.random.RandomState(seed)
    pages = [max(0, -(-s // page)) for s, _ in lens]
    n_blocks = sum(pages) + 3
    order = rs.permutation(n_blocks)
    k, v = make_cache(n_blocks, page, kv_heads, d, dtype, seed, layout)
    width = width or max(max(pages), 1)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, (s, n) in enumerate(lens):
        table[b, : pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        if poison and s > 0:
            if s % page:
                k[int(table[b, s // page]), s % page:] = math.nan
                v[int(table[b, s // page]), s % page:] = math.nan
            if window:
                gone = max(0, s - n - window + 1) // page
                for i in range(gone):
                    k[int(table[b, i])] = math.nan
                    v[int(table[b, i])] = math.nan
                table[b, :gone] = -1
    if poison:
        for i in order[at:]:
            k[int(i)] = math.nan
            v[int(i)] = math.nan
    starts = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
    T = int(starts[-1]) + pad
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.empty((T, heads, d), dtype=dtype, device="cuda").normal_(generator=g)
    return dict(q=q, k=k, v=v, table=torch.from_numpy(table).cuda(), q_start=torch.from_numpy(starts).cuda(),
                seq=torch.tensor([s for s, _ in lens], dtype=torch.int32, device="cuda"), lens=lens, window=window)


def attention(s, scale=None):
    """(out, lse, sum_j p_j |v_j|) in float64: the formula, request by request."""
    q, k, v = s["q"], s["k"], s["v"]
    T, heads, d = q.shape
    page, kv_heads = k.shape[1], k.shape[2]
    group, scale = heads // kv_heads, scale or 1.0 / math.sqrt(d)
    out = torch.zeros((T, heads, d), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device="cuda")
    table, t0 = s["table"].cpu().numpy(), 0
    for b, (seq, n) in enumerate(s["lens"]):
        first = max(0, seq - n - s["window"] + 1) if s["window"] else 0
        if n and seq > first:
            j = np.arange(first, seq)
            blk = torch.from_numpy(table[b, j // page].astype(np.int64)).cuda()
            off = torch.from_numpy(j % page).cuda()
            kk = k[blk, off].double().repeat_interleave(group, 1)
            vv = v[blk, off].double().repeat_interleave(group, 1)
            dots = torch.einsum("thd,jhd->htj", q[t0:t0 + n].double(), kk) * scale
            pos = torch.arange(seq - n, seq, device="cuda")[:, None]
            key = torch.from_numpy(j).cuda()[None, :]
            hidden = key > pos
            if s["window"]:
                hidden = hidden | (key <= pos - s["window"])
            dots = dots.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(dots, -1)
            p = torch.exp(dots - torch.where(z.isinf(), 0.0, z)[..., None])
            out[t0:t0 + n] = torch.einsum("htj,jhd->thd", p, vv)
            mag[t0:t0 + n] = torch.einsum("htj,jhd->thd", p, vv.abs())
            lse[t0:t0 + n] = z.T
        t0 += n
    return out, lse, mag


def check_attention(out, lse, ref, what=""):
    """Each weight is rounded once to the type (half a step of it), so is the
    output; scores, exponentials and sums are in fp32: 2^-14 of the sum of
    magnitudes covers a score of 30 off by the rounding of 128 products. lse
    is off by the scores' error alone."""
    o, z, mag = ref
    half = torch.finfo(out.dtype).eps / 2
    # below the type's smallest normal value the step is absolute
    tol = (half + 2.0 ** -14) * mag + half * o.abs() + torch.finfo(out.dtype).tiny * half * 2
    err = (out.double() - o).abs()
    assert torch.isfinite(out).all(), what
    assert (err <= tol).all(), (what, float((err / tol.clamp_min(1e-300)).max()))
    if lse is not None:
        assert torch.equal(lse.isinf(), z.isinf()), what
        assert (torch.where(z.isinf(), 0.0, lse.double() - z).abs() <= 2.0 ** -13).all(), what


def sample_row(x, u, T=1.0, k=0, p=1.0, mp=0.0):
    """(token, prob, margin): the rules in float64; margin is how near u, or
    top_p, comes to a border at which the answer changes, as a share of the
    mass."""
    x = np.array(x, np.float64)
    x[np.isnan(x)] = -np.inf
    top = x.max()
    if top == -np.inf:
        return -1, 0.0, 1.0
    if not T > 0:
        return int(np.argmax(x)), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        d = np.where(x == top, 0.0, top - x)
    w = np.exp(-d / T)
    order = np.argsort(-x, kind="stable")
    margin = 1.0
    n = len(x) if k <= 0 else min(k, len(x))
    if p < 1:
        c = np.cumsum(w[order[:n]])
        goal = p * c[-1]
        margin = np.abs(c - goal).min() / c[-1]
        n = min(n, max(1, int(np.searchsorted(c, goal, side="left")) + 1))
    kept = np.zeros(len(x), bool)
    kept[order[:n]] = True
    kept &= w >= min(mp, 1.0)
    c = np.cumsum(np.where(kept, w, 0.0))
    goal = min(max(u, 0.0), 1.0) * c[-1]
    token = min(int(np.searchsorted(c, goal, side="right")), int(np.nonzero(kept)[0][-1]))
    margin = min(margin, np.abs(c[kept] - goal).min() / c[-1] if 0 < u < 1 else 1.0)
    return token, w[token] / c[-1], margin
