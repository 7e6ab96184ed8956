"""moe_sample against the rules in float64 (tests/paged_util.py). Masses are
sums of terms with a relative error of some 2^-23, so the cumulated mass is
off by far less than 2^-20 of the total: a row whose u (or top_p) comes that
near to a border may take the neighbour."""
import math

import numpy as np
import pytest
import torch

from paged_util import sample_row

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from moe_decode_gb300 import build
    build.build()
    from moe_decode_gb300 import api as a
    return a


def run(api, logits, u, **settings):
    M = logits.shape[0]
    tokens = torch.full((M,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((M,), math.nan, device="cuda")
    f = {n: (None if v is None else torch.as_tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32).expand(M).contiguous().cuda())
         for n, v in settings.items()}
    api.sample(logits, torch.as_tensor(u, dtype=torch.float32).expand(M).contiguous().cuda(), tokens, probs=probs, **f)
    assert api.last_launch_count() == 1
    return tokens.cpu().numpy(), probs.cpu().numpy(), {n: (None if v is None else v.cpu().numpy()) for n, v in f.items()}


def check(api, logits, u, least=0.9, **settings):
    tokens, probs, f = run(api, logits, u, **settings)
    u = np.broadcast_to(np.asarray(u, np.float32), (logits.shape[0],))
    at = lambda n, r, off: off if f.get(n) is None else f[n][r].item()  # noqa: E731
    clear = 0
    for r, row in enumerate(logits.double().cpu().numpy()):
        want, prob, margin = sample_row(row, float(u[r]), at("temperature", r, 1.0), at("top_k", r, 0), at("top_p", r, 1.0),
                                        at("min_p", r, 0.0))
        if margin > 2.0 ** -20:
            clear += 1
            assert tokens[r] == want, (r, tokens[r], want, margin)
            # a term's error and the rounding of the answer to fp32
            assert abs(probs[r] - prob) <= 2.0 ** -20 * prob, (r, probs[r], prob)
    assert clear >= least * len(u)


def logits_of(M, V, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((M, V), device="cuda").normal_(0, spread, generator=g)
    hot = torch.randint(0, V, (M, 20), device="cuda", generator=g)
    x.scatter_add_(1, hot, torch.empty((M, 20), device="cuda").normal_(5, 2, generator=g))
    return x.to(dtype), torch.rand(M, device="cuda", generator=g).cpu()


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.0),
            dict(top_k=1), dict(temperature=1.3, top_k=1000, top_p=0.95), dict(top_k=7, top_p=0.5, min_p=0.2),
            dict(temperature=0.05, top_p=0.99), dict(temperature=8.0, top_p=0.7), dict(temperature=30.0, top_k=20000, top_p=0.999)]


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 50257])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", SETTINGS, ids=lambda d: "-".join("%s%g" % p for p in d.items()) or "plain")
def test_settings(api, V, dtype, settings):
    x, u = logits_of(5, V, V + len(settings), dtype)
    # (no count of clear rows here: top_p 0.999 of 20,000 nearly equal masses
    # ends within 2^-20 of a border in every row)
    check(api, x, u, least=0.0, **settings)


@pytest.mark.parametrize("M,V", [(1, 157184), (16, 157184), (40, 33333), (200, 3001), (1, 720896), (3, 131073)])
def test_rows_and_vocabularies(api, M, V):
    rs = np.random.RandomState(M)
    x, u = logits_of(M, V, M)
    check(api, x, u, least=0.8, temperature=rs.choice([0.0, 0.6, 1.0, 1.5], M), top_k=rs.choice([0, 1, 20, 1000, V, V + 5], M),
          top_p=rs.choice([1.0, 0.5, 0.95], M), min_p=rs.choice([0.0, 0.01], M))


def test_rows_at_any_stride_and_alignment(api):
    base, u = logits_of(6, 5003, 3)
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.full((6, 5011), 99.0, dtype=dtype, device="cuda")
        wide[:, 3:5006] = base.to(dtype)
        check(api, wide[:, 3:5006], u, top_p=0.9)


@pytest.mark.parametrize("n", [1, 700, 1025, 5000, 40000])
@pytest.mark.parametrize("settings", [dict(top_k=3), dict(top_k=1500), dict(top_p=0.37), dict(top_k=4000, top_p=0.61), dict()], ids=str)
def test_ties_take_the_lower_index(api, n, settings):
    """n equal logits above a few others: the order among them is the index."""
    x = torch.full((4, 60000), -3.0, device="cuda")
    x[:, 100:100 + n] = 2.5
    x[1, 50] = 4.0
    x[2, 59999] = 2.75
    x[3] = 1.0
    check(api, x, [0.2, 0.7, 0.999, 0.41], least=0.5, **settings)


def test_infinities_and_nan(api):
    x = torch.randn((6, 2000), device="cuda")
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 5::7] = math.nan
    x[2, 6::7] = -math.inf
    x[3, [40, 900, 1500]] = math.inf
    x[4] = -math.inf
    x[4, 1234] = -1e30
    x[5, :1000] = -math.inf
    x[5, 1000:] = -0.0
    x[5, 1500] = 0.0
    for settings in (dict(), dict(temperature=0.0), dict(top_k=2), dict(top_k=1999, top_p=0.5), dict(top_p=0.3, min_p=0.5)):
        for u in (0.0, 0.4, 0.99):
            check(api, x, u, least=0.5, **settings)
    tokens, probs, _ = run(api, x, 0.5)
    assert tokens[0] == tokens[1] == -1 and probs[0] == probs[1] == 0
    assert tokens[3] == 900 and abs(probs[3] - 1 / 3) < 1e-6 and tokens[4] == 1234 and probs[4] == 1


def test_random_numbers_at_and_beyond_their_ends(api):
    x, _ = logits_of(6, 3000, 8)
    want = [0, 0, 2999, 2999, 0, 2999]
    tokens, _, _ = run(api, torch.zeros_like(x), [0.0, -1.0, 1.0, 7.0, math.nan, float(np.nextafter(np.float32(1), np.float32(0)))])
    assert tokens.tolist() == want
    x[:, 2000:] = -math.inf
    tokens, _, _ = run(api, x, 1.0, top_p=0.9)
    assert (tokens < 2000).all()


def test_settings_beyond_their_ends(api):
    x, u = logits_of(3, 3000, 9)
    plain = run(api, x, u)[0]
    for settings in (dict(top_k=-5), dict(top_k=1 << 30), dict(top_p=1.0), dict(top_p=5.0), dict(min_p=-1.0), dict(temperature=1.0)):
        assert (run(api, x, u, **settings)[0] == plain).all()
    best = x.argmax(1).cpu().numpy()
    for settings in (dict(temperature=-1.0), dict(temperature=math.nan), dict(top_p=0.0), dict(top_p=-3.0), dict(min_p=1.0),
                     dict(min_p=9.0), dict(temperature=1e-35), dict(top_k=1)):
        assert (run(api, x, u, **settings)[0] == best).all(), settings
    tokens, probs, _ = run(api, x, 0.5, temperature=math.inf)
    assert (tokens == 1500).all() and np.allclose(probs, 1 / 3000, rtol=1e-6)


def test_frequencies_follow_the_masses(api):
    """20,000 rows of one distribution with evenly spread u: each token's
    count is its mass times the rows, to a row or two."""
    x = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -math.inf, 1.5, -2.0], device="cuda")
    n = 20000
    u = (torch.arange(n) + 0.5) / n
    tokens, _, _ = run(api, x.expand(n, 8).contiguous(), u, temperature=0.8, top_k=6)
    w = np.exp(x.cpu().numpy().astype(np.float64) / 0.8)
    w[[5, 7]] = 0
    assert np.abs(np.bincount(tokens, minlength=8) - n * w / w.sum()).max() <= 2


def test_same_token_on_any_split(api):
    """Rows of one call and each row by itself go over other numbers of CTAs."""
    x, u = logits_of(40, 20011, 12)
    together = run(api, x, u, top_p=0.93, temperature=1.1)
    for r in range(0, 40, 7):
        alone = run(api, x[r:r + 1], u[r:r + 1], top_p=0.93, temperature=1.1)
        assert alone[0][0] == together[0][r] and alone[1][0] == together[1][r]


@pytest.mark.parametrize("depth", [12.0, 18.0, 22.0, 26.0])
def test_top_p_ends_among_very_small_masses(api, depth):
    """One token far above hundreds of thousands whose masses are a few units of
    the fixed point each: the run that reaches top_p ends among them."""
    V = 700000
    g = torch.Generator(device="cuda").manual_seed(int(depth))
    x = -depth - torch.rand((4, V), device="cuda", generator=g) * 2.0
    x[:, 4321] = 0.0
    w = torch.exp(x.double())
    share = (w.sum(1) - 1) / w.sum(1)  # of the many
    top_p = (1 - share * torch.tensor([0.2, 0.5, 0.9, 0.999], device="cuda", dtype=torch.float64)).float().cpu()
    tokens, probs, _ = run(api, x, torch.full((4,), 0.9999999), top_p=top_p)
    for r in range(4):
        want, prob, margin = sample_row(x[r].double().cpu().numpy(), float(np.float32(0.9999999)), p=float(top_p[r]))
        if margin > 2.0 ** -20:
            assert tokens[r] == want and abs(probs[r] - prob) <= 2.0 ** -20 * prob, (r, tokens[r], want)
        else:  # within what the masses are known to: some member near the border
            assert 0 <= tokens[r] < V


@pytest.mark.parametrize("settings", [dict(top_p=0.9), dict(top_k=50, top_p=0.9, min_p=0.01), dict(top_k=1000, top_p=0.5)], ids=str)
def test_the_same_on_every_call(api, settings):
    """Rows over 8 and 16 CTAs, 3,000 calls beside another stream's work, which
    shifts the CTAs of a row against each other: the order in which they reach
    each other's memory must not show."""
    rows = [logits_of(M, V, 90 + M, dtype, spread) for M, V, dtype, spread in
            ((14, 49633, torch.bfloat16, 0.01), (27, 38039, torch.float32, 3.0), (5, 157184, torch.float32, 2.0))]
    side, noise = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda")
    for x, u in rows:
        M = x.shape[0]
        f = {n: torch.full((M,), v, device="cuda").to(torch.int32 if n == "top_k" else torch.float32) for n, v in settings.items()}
        u = u.cuda()
        first, tokens = torch.empty(M, dtype=torch.int32, device="cuda"), torch.empty(M, dtype=torch.int32, device="cuda")
        p0, probs = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        api.sample(x, u, first, probs=p0, **f)
        differ = torch.zeros((), dtype=torch.int64, device="cuda")
        for i in range(1000):
            if i % 4 == 0:
                with torch.cuda.stream(side):
                    noise = noise @ noise * 1e-3
            api.sample(x, u, tokens, probs=probs, **f)
            differ += ((tokens != first) | (probs != p0)).sum()
        torch.cuda.synchronize()
        assert differ.item() == 0


def test_equal_logits_have_equal_shares(api):
    """Hundreds of thousands of equal logits under one larger: the share of each
    is 1 / (n + 1 / w). The numerator is one mass and the denominator the sum of
    many, which must be the same number: what is left are three roundings to
    fp32, and the mass's own error in what the larger one adds."""
    n, M = 700000, 32
    t = torch.linspace(4.0, 16.0, M, dtype=torch.float64)
    T = torch.linspace(0.3, 3.1, M).roll(7)
    x = torch.empty((M, n + 1), device="cuda")
    low = (-t * math.log(2) * T.double()).float()
    x[:] = low.cuda()[:, None]
    x[:, 0] = 0.0
    tokens, probs, _ = run(api, x, 0.9, temperature=T)
    w = torch.exp(low.double() / T.double()).numpy()
    want = 1 / (n + 1 / w)
    assert (tokens > 0).all()
    err = np.abs(probs / want - 1)
    assert (err <= 3 * 2.0 ** -24 + 2.0 ** -21 / w * want).all(), err.max() * 2.0 ** 24


def test_a_token_at_every_u_below_one(api):
    """The mass of a row lies in its last few logits and u is the largest fp32
    below 1: every row gets one of them."""
    M, V, hot = 2000, 19976, 44
    t = 4 + 4 * torch.rand(M, generator=torch.Generator().manual_seed(1))
    T = 0.2 + 2 * torch.rand(M, generator=torch.Generator().manual_seed(2))
    x = torch.full((M, V), -math.inf, device="cuda")
    x[:, V - hot:] = (-t * math.log(2) * T).cuda()[:, None]
    x[:, 0] = 0.0
    u = float(np.nextafter(np.float32(1), np.float32(0)))
    for settings in (dict(), dict(top_k=hot + 1), dict(top_p=0.999), dict(min_p=1e-4)):
        tokens, probs, _ = run(api, x, u, temperature=T, **settings)
        assert (tokens >= V - hot).all() and (tokens < V).all() and (probs > 0).all(), (settings, tokens.min())


def test_more_rows_than_20_bits(api):
    M = (1 << 20) + 37
    x = torch.full((M, 8), -1.0, device="cuda")
    want = torch.arange(M, device="cuda") % 8
    x.scatter_(1, want[:, None], 60.0)
    tokens, probs, _ = run(api, x, 0.5, temperature=1.0)
    assert (tokens == want.cpu().numpy()).all() and (probs == 1.0).all()


def test_settings_that_are_nan(api):
    """A NaN top_p or min_p is off, a NaN temperature takes the largest."""
    x, u = logits_of(9, 5000, 15)
    plain = run(api, x, u, temperature=0.9)
    for settings in (dict(top_p=math.nan), dict(min_p=math.nan), dict(top_p=math.nan, min_p=math.nan)):
        got = run(api, x, u, temperature=0.9, **settings)
        assert (got[0] == plain[0]).all() and (got[1] == plain[1]).all(), settings
    assert (run(api, x, u, temperature=math.nan, top_p=math.nan)[0] == x.argmax(1).cpu().numpy()).all()


@pytest.mark.parametrize("V", [31, 1000, 50257])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", SETTINGS[:-1], ids=lambda d: "-".join("%s%g" % p for p in d.items()) or "plain")
def test_settings_on_clear_rows(api, V, dtype, settings):
    """test_settings with a count of the rows that were compared. The worst is
    top_p among some 50,000 masses of 10^-5: a border comes within 2^-20 in one
    row of five."""
    x, u = logits_of(64, V, 3 * V + len(settings), dtype)
    check(api, x, u, least=0.5, **settings)


# (at a depth of 26 the small masses together are known to a tenth, and hold
# some twenty fp32 u: one share of them alone can be told)
@pytest.mark.parametrize("depth,dropped", [(d, f) for d in (12.0, 18.0, 22.0) for f in (0.2, 0.5, 0.9)] + [(26.0, 0.5)])
def test_top_p_keeps_what_reaches_it_of_very_small_masses(api, depth, dropped):
    """The rows of test_top_p_ends_among_very_small_masses at 256 u that fall
    among the small masses. The sums are known to `known` (2^-22 of a mass and a
    unit of 2^-42 each), so no token may lie further behind the border of the
    kept run than twice that (the run's mass and its goal), nor away from where u
    points by more than what the border's place and the sums together move."""
    V, M = 700000, 256
    g = torch.Generator(device="cuda").manual_seed(int(depth))
    x = -depth - torch.rand(V, device="cuda", generator=g) * 2.0
    x[4321] = 0.0
    w = torch.exp(x.double()).cpu().numpy()
    total, small = w.sum(), w.sum() - 1
    top_p = float(np.float32(1 - dropped * small / total))
    order = np.argsort(-x.cpu().numpy(), kind="stable")
    before = np.cumsum(w[order]) - w[order]  # in the order of the run
    keep = int(np.searchsorted(before, top_p * total, side="left"))
    place = np.empty(V)
    place[order] = before
    kept = np.zeros(V, bool)
    kept[order[:keep]] = True
    cdf = np.cumsum(np.where(kept, w, 0.0))
    known, one = small * 2.0 ** -22 + V * 2.0 ** -42, w[order[1]]
    assert total - top_p * total > 3 * known  # there is something that must not be taken
    # u over the small masses behind the large one
    u = (1 - (1 - cdf[4321] / cdf[-1]) * (torch.arange(M, dtype=torch.float64) + 0.5) / M).float().clamp_max(1 - 2.0 ** -24)
    tokens, probs, _ = run(api, x.expand(M, V).contiguous(), u, top_p=top_p)
    assert (tokens != 4321).sum() >= 0.7 * M and len(np.unique(tokens)) >= 8
    assert (place[tokens] <= top_p * total + 2 * known).all()
    goal = u.double().numpy() * cdf[-1]
    slack = 6 * known + 2 * one
    assert (cdf[tokens] - np.where(kept[tokens], w[tokens], 0.0) <= goal + slack).all()
    assert (cdf[tokens] >= goal - slack).all()
    share = w[tokens] / cdf[-1]
    assert (np.abs(probs - share) <= share * 2.0 ** -20 + share * slack + 2.0 ** -42).all()
