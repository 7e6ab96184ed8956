"""Plain references, in 64 bits, of rotary positions and of the cache of 8-bit
values."""
import math

import numpy as np
import torch


def e4m3_values():
    """The 127 finite magnitudes by code: 3 bits of mantissa, exponent bias 7."""
    return np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def exponent(x):
    """The least e >= -127 with max |x| <= 448 2^e of each row of the last dimension (float64 array, finite)."""
    top = np.abs(x).max(-1)
    m, e = np.frexp(top)  # m in [0.5, 1): 448 = 0.875 * 2^9
    return np.where(top > 0, np.maximum(e - 9 + (m > 0.875), -127), -127)


def quantise(x):
    """(codes, bytes) of float64 rows: by search in the table, a tie to the even code; a row that is not finite gets byte 255 and codes 0."""
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[..., None], x, 0.0)
    e = exponent(x)
    y = x / 2.0 ** e[..., None]
    v = e4m3_values()
    hi = np.searchsorted(v, np.abs(y)).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    near = np.where(v[hi] - np.abs(y) < np.abs(y) - v[lo], hi, lo)
    near = np.where((v[hi] - np.abs(y) == np.abs(y) - v[lo]) & (hi % 2 == 0), hi, near)
    codes = near + 128 * np.signbit(y)
    return np.where(fine[..., None], codes, 0).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def dequantise(codes, byte):
    """float64 values of codes [..., d] with bytes [...]."""
    v = np.concatenate([e4m3_values(), [np.nan]])
    x = v[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return np.where((byte == 255)[..., None], np.nan, x * 2.0 ** (byte.astype(np.float64) - 127)[..., None])


def make_cache8(api, n_blocks, page, heads, d, layout="bthd", fill=None):
    """A KvCache8 over the layout's own buffers, filled with random codes (seed `fill`) or 0xAA."""
    def one():
        shape = (n_blocks, heads, page, d) if layout == "bhtd" else (n_blocks, page, heads, d)
        t = torch.full(shape, 0xAA, dtype=torch.uint8, device="cuda")
        return t.transpose(1, 2) if layout == "bhtd" else t

    if layout == "pair":  # K and V of a block side by side
        both = torch.full((n_blocks, 2, page, heads, d), 0xAA, dtype=torch.uint8, device="cuda")
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = one(), one()
    ks, vs = (torch.full((n_blocks, heads, page), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    return api.KvCache8(k, v, ks, vs)


def by_slot(cache):
    """codes [slots, heads, d] and bytes [slots, heads] of K and V as numpy arrays."""
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        out.append((x.cpu().numpy().reshape(-1, *x.shape[2:]), s.transpose(1, 2).cpu().numpy().reshape(-1, x.shape[2])))
    return out


def rotate(x, positions, turns, rotary_dim, interleaved, scale):
    """x [T, heads, d] (float64 tensor) turned; turns: int64 tensor of 2^-64 turns a position, positions below 0: as they are. Also the
    magnitudes |first| + |second| of each pair, in both of its places."""
    phase = positions.long()[:, None].cpu().numpy().astype(np.uint64) * turns.cpu().numpy().view(np.uint64)[None]  # modulo 2^64
    angle = torch.from_numpy(phase.astype(np.float64) * (2 * math.pi / 2.0 ** 64)).to(x.device)[:, None]
    c, s = angle.cos() * scale, angle.sin() * scale
    i = torch.arange(rotary_dim // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    mag[..., first] = mag[..., second] = (a.abs() + b.abs()) * abs(scale)
    real = (positions >= 0)[:, None, None]
    return torch.where(real, y, x), mag


def make_step8(api, lens, page, heads, kv_heads, d, dtype, seed, layout="bthd", window=0, pad=0, spread=(1.0, 1.0)):
    """Inputs of paged_attention over a KvCache8 for requests lens = [(seq, new), ...]: tokens of sizes 2^normal(0, spread) in keys and
    values; what no row may read is poisoned (codes of NaN, byte 255, table entries -1). k and v hold the values in 64 bits."""
    rs = np.random.RandomState(seed)
    pages = [max(0, -(-s // page)) for s, _ in lens]
    n_blocks = sum(pages) + 3
    order = rs.permutation(n_blocks)
    cache = make_cache8(api, n_blocks, page, kv_heads, d, layout)
    cache.k.fill_(0x7F)
    cache.v.fill_(0xFF)
    cache.k_scale.fill_(255)
    cache.v_scale.fill_(255)
    table = np.full((len(lens), max(max(pages), 1)), -1, np.int32)
    held = np.zeros((n_blocks, page), bool)
    at = 0
    for b, (s, n) in enumerate(lens):
        table[b, : pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        gone = max(0, s - n - window + 1) // page if window else 0
        for i in range(gone, pages[b]):
            held[table[b, i], : min(page, s - i * page)] = True
        table[b, :gone] = -1
    values = []
    for x, scale, by in ((cache.k, cache.k_scale, spread[0]), (cache.v, cache.v_scale, spread[1])):
        v = rs.randn(n_blocks, page, kv_heads, d) * 2.0 ** (rs.randn(n_blocks, page, kv_heads, 1) * by)
        codes, byte = quantise(v)
        on = torch.from_numpy(held).cuda()
        x[on] = torch.from_numpy(codes).cuda()[on]
        scale.transpose(1, 2)[on] = torch.from_numpy(byte).cuda()[on]
        values.append(torch.from_numpy(dequantise(codes, byte)).cuda())
    starts = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.empty((int(starts[-1]) + pad, heads, d), dtype=dtype, device="cuda").normal_(generator=g)
    return dict(q=q, cache=cache, k=values[0], v=values[1], table=torch.from_numpy(table).cuda(), q_start=torch.from_numpy(starts).cuda(),
                seq=torch.tensor([s for s, _ in lens], dtype=torch.int32, device="cuda"), lens=lens, window=window)


def check_attention8(out, lse, ref, most_keys, what=""):
    """Each weight is rounded once to fp16 (half a step, 2^-11 of it), the output once to its type; scores, exponentials and sums are in
    fp32 (2^-14 of the sum of magnitudes, as over a 16-bit cache). Below 2^-14 a weight's step is absolute, 2^-25 where the row's largest
    (weight times power of two of the values, which `mag` holds at least half of in its largest element) is at least 2^11: 448 * 2^-36 of
    it for each of the keys."""
    o, z, mag = ref
    half = torch.finfo(out.dtype).eps / 2
    tol = (2.0 ** -11 + 2.0 ** -14) * mag + half * o.abs() + torch.finfo(out.dtype).tiny * half * 2
    tol = tol + most_keys * 2.0 ** -27 / 224 * mag.amax(-1, keepdim=True)
    err = (out.double() - o).abs()
    assert torch.isfinite(out).all(), what
    assert (err <= tol).all(), (what, float((err / tol.clamp_min(1e-300)).max()))
    if lse is not None:
        assert torch.equal(lse.isinf(), z.isinf()), what
        assert (torch.where(z.isinf(), 0.0, lse.double() - z).abs() <= 2.0 ** -13).all(), what
