"""Plain references of trees of drafted tokens: masks and positions, and
attention under them in 64 bits."""
import math

import numpy as np
import torch


def random_parents(rs, n):
    """Each token continues one of the few before it, or the context."""
    return [-1 if i == 0 or rs.rand() < 0.15 else int(max(0, i - 1 - rs.geometric(0.4) + 1)) for i in range(n)]


def plan(parents, lens):
    """(masks, positions) of requests lens = [(seq, new), ...]: each path walked up to its root. parents: by request."""
    masks, positions = [], []
    for up, (seq, n) in zip(parents, lens):
        for i in range(n):
            if n > 64:
                masks.append(-1)
                positions.append(seq - n + i)
                continue
            path, j = 0, i
            while j >= 0:
                path |= 1 << j
                j = up[j]
            masks.append(path - (1 << 64) if path >> 63 else path)
            positions.append(seq - n + bin(path).count("1") - 1)
    return masks, positions


def attention(s, masks, scale=None):
    """paged_util.attention with masks (whole numbers, one a token row)."""
    q, k, v = s["q"], s["k"], s["v"]
    T, heads, d = q.shape
    page, kv_heads = k.shape[1], k.shape[2]
    group, scale = heads // kv_heads, scale or 1.0 / math.sqrt(d)
    out = torch.zeros((T, heads, d), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device="cuda")
    table, t0 = s["table"].cpu().numpy(), 0
    for b, (seq, n) in enumerate(s["lens"]):
        if n and seq > 0:
            j = np.arange(seq)
            blk = torch.from_numpy(table[b, j // page].astype(np.int64)).cuda()
            off = torch.from_numpy(j % page).cuda()
            kk = k[blk, off].double().repeat_interleave(group, 1)
            vv = v[blk, off].double().repeat_interleave(group, 1)
            dots = torch.einsum("thd,jhd->htj", q[t0:t0 + n].double(), kk) * scale
            ctx = seq - n
            hidden = np.zeros((n, seq), bool)
            for i in range(n):
                hidden[i, max(0, ctx + i + 1):] = True
                if n <= 64:
                    for a in range(i + 1):
                        if ctx + a >= 0 and not (masks[t0 + i] >> a) & 1:
                            hidden[i, ctx + a] = True
            dots = dots.masked_fill(torch.from_numpy(hidden).cuda(), -math.inf)
            z = torch.logsumexp(dots, -1)
            p = torch.exp(dots - torch.where(z.isinf(), 0.0, z)[..., None])
            out[t0:t0 + n] = torch.einsum("htj,jhd->thd", p, vv)
            mag[t0:t0 + n] = torch.einsum("htj,jhd->thd", p, vv.abs())
            lse[t0:t0 + n] = z.T
        t0 += n
    return out, lse, mag
