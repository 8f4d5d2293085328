"""Tokens drawn from logits on the GPU against the definition in 64 bits, a row at a time on the CPU.

A token has to be the definition's.  Weights are formed to 2^-30 of themselves and summed exactly, so the sums that a
border is compared with are off by at most 2^-30 of the whole (plus 2^18 weights that count as zero, 2^-48 each): another
token is right too if the drawn number lies within EDGE = 2^-29 of the border between them.  logprobs: the logarithm of a share
off by 2^-29, then rounded to f32 (2^-24 of itself).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EDGE = 2.0 ** -29


@pytest.fixture(scope="module")
def tk():
    import top_selection_prof_gb300 as m
    return m


def f32(v):
    return float(np.float32(v))


def kept_of(x, temperature, top_k, top_p, min_p):
    """(tokens in their order, sums of their weights up to each) of what is kept of one row, from the definition."""
    x = x.double().numpy()
    may = np.nonzero(x > -np.inf)[0]      # (NaN compares false)
    if may.size == 0:
        return may, np.zeros(0)
    order = may[np.argsort(-x[may], kind="stable")]
    if not temperature > 0:
        return order[:1], np.ones(1)
    top = x[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / temperature))
    keep = w >= min(max(min_p, 0.0), 1.0)
    order, w = order[keep], w[keep]
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    cum = np.array(np.cumsum(w.astype(np.longdouble)), dtype=np.longdouble)
    if top_p < 1:
        n = int(np.searchsorted(cum, max(top_p, 0.0) * cum[-1])) + 1
        order, cum = order[:n], cum[:n]
    return order, cum.astype(np.float64)


def check(x, u, tokens, logprobs, temperature, top_k, top_p, min_p):
    x, u = x.float().cpu(), u.cpu()
    tokens, logprobs = tokens.cpu(), logprobs.double().cpu()
    rows = x.shape[0]

    def each(v):
        return v.cpu().tolist() if isinstance(v, torch.Tensor) else [v if isinstance(v, int) else f32(v)] * rows

    params = list(zip(each(temperature), each(top_k), each(top_p), each(min_p)))
    for r in range(rows):
        order, cum = kept_of(x[r], *params[r])
        got = int(tokens[r])
        if order.size == 0:
            assert got == -1 and logprobs[r] == -math.inf, r
            continue
        at = np.nonzero(order == got)[0]
        assert at.size == 1, "row %d: %d is not kept" % (r, got)
        i = int(at[0])
        low, high = (cum[i - 1] if i else 0.0) / cum[-1], cum[i] / cum[-1]
        v = min(max(float(u[r]), 0.0), 1.0)
        inside = low <= v < high or (i == 0 and v <= low) or (i == order.size - 1 and v >= high)
        assert inside or low - EDGE <= v <= high + EDGE, "row %d: %d at [%.12g, %.12g), drawn by %.12g" % (r, got, low, high, v)
        share = math.log(high - low) if high > low else -math.inf
        # (high - low loses bits of its own: 2^-52 of the sums before it)
        room = 2.0 ** -23 * abs(share) + 2.0 ** -28 + 2.0 ** -50 / max(high - low, 1e-300)
        assert abs(float(logprobs[r]) - share) <= room, "row %d: logprob %g, %g expected" % (r, float(logprobs[r]), share)


def logits(rows, n, dtype, seed, spread=2.0, peaks=24):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g) * spread
    if peaks:
        x.scatter_add_(1, torch.randint(0, n, (rows, peaks), generator=g), 12 * torch.rand(rows, peaks, generator=g) * torch.rand(rows, 1, generator=g))
    return x.to(dtype).cuda(), torch.rand(rows, generator=g).cuda()


def draw(tk, x, u, **kw):
    a = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    a.update(kw)
    tokens, logprobs = tk.sample(x, u, **a)
    assert tokens.dtype == torch.int64 and logprobs.dtype == torch.float32 and tokens.shape == logprobs.shape == u.shape
    check(x, u, tokens, logprobs, **a)
    return tokens, logprobs


FILTERS = [dict(), dict(top_k=1), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=40, top_p=0.8, min_p=0.01),
           dict(temperature=0.0), dict(temperature=0.3, top_p=0.5), dict(temperature=3.0), dict(temperature=20.0, top_p=0.97),
           dict(top_k=5000, top_p=0.99), dict(top_p=0.0), dict(min_p=1.0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 2, 7, 1000, 8191, 40013])
def test_filters(tk, n, dtype):
    x, u = logits(9, n, dtype, n)
    for kw in FILTERS:
        draw(tk, x, u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [300, 2239, 2240, 2241, 2600])
def test_rows_around_what_one_block_holds(tk, n, dtype):
    x, u = logits(5, n, dtype, n)
    x[1, ::3], x[2, :] = -math.inf, x[2, 0].item()
    for kw in (dict(), dict(top_p=0.9, min_p=0.01), dict(top_k=n - 1), dict(temperature=1e30), dict(temperature=3e38, top_k=n - 1, top_p=0.5),
               dict(temperature=1e38, top_k=7)):
        draw(tk, x, u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 131072), (3, 262144), (40, 70001), (170, 12289)])
def test_sizes(tk, rows, n, dtype):
    x, u = logits(rows, n, dtype, rows)
    for kw in (dict(), dict(top_p=0.95), dict(top_k=64, top_p=0.9), dict(temperature=8.0)):
        draw(tk, x, u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(160, 131073), (5, 150_001), (160, 200_003), (200, 262_144)])
def test_rows_that_take_two_blocks_or_more(tk, rows, n, dtype):
    """More tokens than one block adds up, in a few rows and in more than run at once, with filters.  (Rows repeat eight, each with
    its own number.)"""
    few, _ = logits(8, n, dtype, rows)
    x = few.repeat(rows // 8 + 1, 1)[:rows].contiguous()
    u = ((torch.arange(rows) + 0.5) / rows).cuda()
    for kw in (dict(top_p=0.95), dict(top_k=50, top_p=0.9, min_p=0.01), dict(temperature=2.0, min_p=0.02), dict(top_k=n // 2, temperature=4.0)):
        tokens, logprobs = tk.sample(x, u, **kw)
        some = slice(0, rows, max(1, rows // 10))
        check(x[some], u[some], tokens[some], logprobs[some], **{**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw})
        again = tk.sample(few[:rows], u[:8], **kw)      # (more blocks a row: the same bits)
        assert torch.equal(again[0], tokens[:8]) and torch.equal(again[1], logprobs[:8])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_flat_and_equal_rows(tk, dtype):
    """One bin holds more tokens than a block searches: equal values, nearly equal ones, two values, a long flat tail."""
    n = 100_000
    g = torch.Generator().manual_seed(5)
    x = torch.zeros(8, n)
    x[1] = -7.5
    x[2] = torch.randn(n, generator=g) * 1e-4
    x[3] = torch.where(torch.rand(n, generator=g) < 0.5, 1.0, 1.0078125)
    x[4, 5] = 30.0
    x[5] = torch.randn(n, generator=g) * 1e-3 - 20
    x[5, 77] = 0.0
    x[6] = torch.arange(n) * 1e-7
    x[7] = torch.randint(0, 3, (n,), generator=g) * 0.001
    x = x.to(dtype).cuda()
    for seed in range(3):
        u = torch.rand(8, generator=g).cuda()
        for kw in (dict(), dict(top_p=0.7), dict(top_k=30_000), dict(top_k=99_999, top_p=0.9), dict(temperature=0.5, min_p=0.9)):
            draw(tk, x, u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_deep_tails(tk, dtype):
    """The drawn token lies 16 and 32 octaves below the likeliest, among tokens whose number makes up for it."""
    n = 200_000
    g = torch.Generator().manual_seed(6)
    x = torch.randn(6, n, generator=g) * 0.05
    for r, top in enumerate((8.0, 12.0, 12.5, 14.0, 23.0, 30.0)):
        x[r, 1000 * r] = top
    x = x.to(dtype).cuda()
    for u in (0.3, 0.9, 0.999, 1 - 2.0 ** -24):
        draw(tk, x, torch.full((6,), u, device="cuda"))
        draw(tk, x, torch.full((6,), u, device="cuda"), top_p=0.999)
        draw(tk, x, torch.full((6,), u, device="cuda"), top_k=150_000)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_deep_head_counts_towards_top_k(tk, dtype):
    """All tokens but one lie 45 to 48 octaves below the likeliest: they weigh next to nothing, and are the first top_k all the same.
    (With u = 1 the last that is kept, to EDGE, may be any that is kept, and none that is not.)"""
    n = 5000
    g = torch.Generator().manual_seed(15)
    x = -math.log(2.0) * (45.05 + 2.9 * torch.rand(6, n, generator=g))
    x[torch.arange(6), torch.randint(0, n, (6,), generator=g)] = 0.0
    x = x.to(dtype).cuda()
    for u in (1.0, 1 - 2.0 ** -24, 0.5):
        for top_k in (2, 40, 300, 1500, 4000):
            draw(tk, x, torch.full((6,), u, device="cuda"), top_k=top_k)
            draw(tk, x, torch.full((6,), u, device="cuda"), top_k=torch.full((6,), top_k, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_rows(tk, dtype):
    """-inf, NaN and the type's lowest value in masked places, rows with one token or none left, infinities."""
    n = 5003
    low = torch.finfo(dtype).min
    x, u = logits(9, n, dtype, 3)
    keep = torch.arange(n, device="cuda") % 97 == 5
    x[0] = -torch.inf
    x[1] = torch.nan
    x[2] = torch.where(keep, x[2], -torch.inf)
    x[3] = torch.where(keep, x[3], torch.nan)
    x[4] = torch.where(keep, x[4], low)
    x[5] = low
    x[6] = -torch.inf
    x[6, 4321] = -3.0
    x[7, 11], x[7, 4000] = torch.inf, torch.inf
    x[8, 17] = torch.finfo(dtype).max
    for kw in (dict(), dict(top_k=20), dict(top_p=0.8), dict(temperature=0.0), dict(min_p=0.1, top_k=3), dict(temperature=1e-30),
               dict(temperature=1e30)):
        tokens, _ = draw(tk, x, u, **kw)
        assert tokens[:2].tolist() == [-1, -1]
        assert int(tokens[6]) == 4321 and int(tokens[7]) in (11, 4000) and int(tokens[8]) == 17 or kw.get("temperature") == 1e30


def test_drawn_numbers_at_their_ends(tk):
    x, _ = logits(8, 3001, torch.float32, 8)
    u = torch.tensor([0.0, 1.0, -1.0, 2.0, torch.nan, 1 - 2.0 ** -24, 2.0 ** -149, 0.5], device="cuda")
    tokens, _ = tk.sample(x, u, top_k=50)
    order = x.sort(dim=1, descending=True, stable=True).indices
    assert torch.equal(tokens[[0, 2, 4, 6]], order[[0, 2, 4, 6], 0]) and torch.equal(tokens[[1, 3]], order[[1, 3], 49])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parameters_by_row(tk, dtype):
    rows, n = 41, 30_011
    x, u = logits(rows, n, dtype, 4)
    g = torch.Generator().manual_seed(9)
    t = (torch.rand(rows, generator=g) * 2).cuda()
    t[3], t[4], t[5] = 0.0, -1.0, torch.nan
    k = torch.randint(-3, 400, (rows,), generator=g).int().cuda()
    p = (torch.rand(rows, generator=g) * 1.2).cuda()
    p[6], p[7] = -0.5, torch.nan
    m = (torch.rand(rows, generator=g) * 0.1 - 0.02).cuda()
    m[8], m[9] = 3.0, torch.nan
    got = tk.sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    plain = dict(top_p=torch.where(p.isnan(), 1.0, p), min_p=torch.where(m.isnan(), 0.0, m), temperature=t, top_k=k)
    check(x, u, *got, **plain)


def test_strided_rows_and_offsets(tk):
    """Rows that start anywhere, and are far apart, give what contiguous ones give."""
    for dtype in (torch.bfloat16, torch.float32):
        x, u = logits(5, 20_001, dtype, 10)
        want = tk.sample(x, u, temperature=0.9, top_p=0.95)
        for offset in range(8):
            big = torch.full((5, 20_033), 50.0, dtype=dtype, device="cuda")
            v = big[:, offset:offset + 20_001]
            v.copy_(x)
            got = tk.sample(v, u, temperature=0.9, top_p=0.95)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_shares_are_the_distributions(tk):
    """4096 draws from one row, evenly spread over [0, 1): every token comes as often as its share says, to one."""
    x, _ = logits(1, 257, torch.float32, 11, peaks=0)
    draws = 4096
    u = (torch.arange(draws, device="cuda") + 0.5) / draws
    tokens, _ = tk.sample(x.expand(draws, -1).contiguous(), u, temperature=1.3)
    count = torch.bincount(tokens, minlength=257).double()
    share = torch.softmax(x[0].double() / f32(1.3), 0) * draws
    assert float((count - share).abs().max()) <= 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(310, 131072), (310, 131073), (160, 262144)])
def test_equal_tokens_in_the_largest_parts(tk, rows, n, dtype):
    """As many equal weights as a block adds up: token floor(u n), with sums that would pass 32 bits if a half were larger."""
    u = ((torch.arange(rows) + 0.5) / rows).cuda()
    x = torch.full((rows, n), -1.25, dtype=dtype, device="cuda")
    tokens, logprobs = tk.sample(x, u)
    assert torch.equal(tokens, (u.double() * n).long())
    assert float((logprobs.double() + math.log(n)).abs().max()) <= 2.0 ** -23 * math.log(n) + 2.0 ** -28
    x[:, 7] = 0.0
    tokens, _ = tk.sample(x, u, top_k=n - 1)
    order = torch.cat([torch.tensor([7]), torch.arange(7), torch.arange(8, n)]).cuda()
    w = torch.full((n - 1,), math.exp(-1.25), dtype=torch.float64, device="cuda")
    w[0] = 1.0
    cum = w.cumsum(0) / w.sum()
    at = torch.searchsorted(cum, u.double(), right=True)
    near = (cum[(at - 1).clamp(min=0)] - u.double()).abs().minimum((cum[at] - u.double()).abs()) < EDGE
    assert bool(((tokens == order[at]) | near).all())


def test_the_same_call_gives_the_same_tokens(tk):
    for dtype in (torch.bfloat16, torch.float32):
        x, u = logits(60, 70_003, dtype, 21)
        for kw in (dict(top_p=0.9), dict(temperature=4.0), dict(top_k=5000, top_p=0.95, min_p=1e-4)):
            first = tk.sample(x, u, **kw)
            for _ in range(5):
                again = tk.sample(x, u, **kw)
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_capture_streams_and_no_rows(tk):
    x, u = logits(7, 50_021, torch.float32, 12)
    y, v = logits(7, 50_021, torch.float32, 13)
    kw = dict(top_k=100, top_p=0.9, min_p=torch.full((7,), 0.001, device="cuda"))
    want = [tk.sample(x, u, **kw), tk.sample(y, v, **kw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tk.sample(x, u, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tk.sample(x, u, **kw)
    x.copy_(y)
    u.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[1][0]) and torch.equal(out[1], want[1][1])
    assert tk.sample(x[:0], u[:0])[0].shape == (0,)


def test_refusals(tk):
    x, u = logits(4, 100, torch.float32, 14)
    for kw in (dict(temperature=-1.0), dict(temperature=math.inf), dict(temperature=math.nan), dict(top_k=-1), dict(top_p=1.5),
               dict(top_p=-0.1), dict(min_p=1.5), dict(min_p=math.nan)):
        with pytest.raises(tk.TopkError) as e:
            tk.sample(x, u, **kw)
        assert e.value.status == -1
    with pytest.raises(tk.TopkError) as e:
        tk.sample(torch.zeros(1, 262145, device="cuda"), u[:1])
    assert e.value.status == -4
    with pytest.raises(ValueError):
        tk.sample(x, u[:3])
    with pytest.raises(ValueError):
        tk.sample(x[0], u[:1])
    with pytest.raises(ValueError):
        tk.sample(x.t(), u)
    with pytest.raises(TypeError):
        tk.sample(x, u.double())
    with pytest.raises(TypeError):
        tk.sample(x, u, top_k=torch.ones(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        tk.sample(x.half(), u)
    with pytest.raises(TypeError):
        tk.sample(x.cpu(), u)
