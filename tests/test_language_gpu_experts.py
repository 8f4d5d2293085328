"""Rows sorted by expert and back on the GPU against plain forms on the CPU in 64 bits.

Moved rows are compared bit for bit.  A product of two bf16 or two f32 values has at most 48 bits, so a gradient that is one
product, and a sum of small whole numbers, are exact in 64 bits and rounded once: bit for bit too.  Other sums of n products
formed in f32 in any order are off by at most n 2^-24 times the sum of their magnitudes, and by the result's own rounding
(half a step: 2^-8 of it for bf16, 2^-24 for f32).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def tk():
    import top_selection_prof_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def routed(tokens, k, experts, seed, dropped=0.1):
    g = gen(seed)
    idx = torch.rand(tokens, experts, generator=g).topk(min(k, experts), 1).indices
    if k > experts:
        idx = torch.randint(0, experts, (tokens, k), generator=g)
    return torch.where(torch.rand(idx.shape, generator=g) < dropped, torch.tensor([-1, experts, -(1 << 40)])[torch.randint(0, 3, idx.shape, generator=g)], idx)


def sort64(idx, experts):
    flat = idx.reshape(-1)
    held = (flat >= 0) & (flat < experts)
    order = torch.where(held, flat, experts).sort(stable=True).indices
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel())
    count = torch.bincount(flat[held], minlength=experts)
    return torch.where(held, place, -1).view(idx.shape), torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)]), order


def check_dispatch(tk, x, idx, experts):
    xs, place, offsets = tk.dispatch(x, idx.cuda(), experts)
    p, o, order = sort64(idx, experts)
    assert torch.equal(place.cpu(), p) and torch.equal(offsets.cpu(), o)
    want = torch.zeros(order.numel(), x.shape[1], dtype=x.dtype)
    m = int(o[-1])
    want[:m] = x.cpu()[order[:m] // idx.shape[1]]
    assert torch.equal(xs.cpu(), want)
    return xs, place, offsets


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,experts,d", [(1, 1, 1, 1), (1, 4, 8, 64), (16, 4, 64, 4096), (33, 3, 7, 65), (128, 8, 256, 72), (1000, 1, 2, 8),
                                                (129, 8, 64, 1001), (700, 6, 60, 257), (5000, 2, 4096, 40), (3, 700, 5, 24), (20_000, 8, 16, 16),
                                                (2048, 12, 4000, 64), (1, 1500, 3, 2000), (300, 5, 1, 128)])
def test_dispatch(tk, tokens, k, experts, d, dtype):
    x = torch.randn(tokens, d, generator=gen(d)).to(dtype).cuda()
    for dropped in (0.0, 0.1, 1.0):
        check_dispatch(tk, x, routed(tokens, k, experts, tokens + k, dropped), experts)


@pytest.mark.parametrize("experts", [1, 31, 32, 318, 319, 320, 321, 511, 1024, 4096])
@pytest.mark.parametrize("tokens,k", [(513, 2), (1024, 1), (1025, 1), (40_000, 4)])
def test_dispatch_around_the_ranks_limits(tk, tokens, k, experts):
    x = torch.randn(tokens, 8, generator=gen(experts)).cuda()
    check_dispatch(tk, x, routed(tokens, k, experts, experts), experts)


def test_dispatch_of_one_expert_and_of_strided_rows(tk):
    for dtype in DTYPES:
        big = torch.randn(3000, 150, generator=gen(1)).to(dtype).cuda()
        for x in (big[:, :128], big[:, 3:131], big[::2, 8:136]):
            idx = torch.full((x.shape[0], 2), 5)
            idx[17, 1], idx[100, 0] = -1, 3
            check_dispatch(tk, x, idx, 9)


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def within(got, want, magnitude, n, dtype):
    bound = n * 2.0 ** -24 * magnitude + half_step(dtype) * want.abs() + 1e-38
    bad = (got.double().cpu() - want).abs() > bound
    assert not bad.any(), "%d outside, first %s" % (int(bad.sum()), bad.nonzero()[:1].tolist())


def places64(place, rows):
    held = (place >= 0) & (place < rows)
    return held, torch.where(held, place, 0)


def combine64(ys, place, w):
    held, at = places64(place, ys.shape[0])
    t = torch.where(held[..., None], ys[at], torch.zeros((), dtype=ys.dtype)) if ys.shape[0] else torch.zeros(*place.shape, ys.shape[1], dtype=ys.dtype)
    return t if w is None else t * w[..., None]


def backward64(dy, ys, place, w):
    held, at = places64(place, ys.shape[0])
    dys, size = torch.zeros_like(ys), torch.zeros_like(ys)
    t, j = held.nonzero(as_tuple=True)
    terms = dy[t] * (1.0 if w is None else w[t, j][:, None])
    dys.index_add_(0, at[t, j], terms)
    size.index_add_(0, at[t, j], terms.abs())
    prod = combine64(ys, place, None) * dy[:, None]
    return dys, size, prod.sum(-1), prod.abs().sum(-1)


CASES = [(1, 1, 1, 1), (1, 8, 8, 4096), (16, 4, 64, 512), (37, 3, 200, 65), (500, 8, 4100, 136), (700, 6, 4200, 1001), (64, 20, 1300, 2500),
         (3, 33, 50, 7), (4000, 2, 8000, 24)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,rows,d", CASES)
def test_combine_and_its_gradients(tk, tokens, k, rows, d, dtype):
    """Places in no order, rows listed never, once or often, places out of range; with and without weights."""
    g = gen(tokens + d)
    for kind in ("once", "any"):
        n = tokens * k
        if kind == "once":
            place = torch.full((n,), -1)
            take = torch.randperm(n, generator=g)[:min(n, rows)]
            place[take] = torch.randperm(rows, generator=g)[:take.numel()]
        else:
            place = (torch.rand(n, generator=g) ** 3 * rows * 1.1).long() - 1
            place[torch.rand(n, generator=g) < 0.02] = 1 << 40
        place = place.view(tokens, k)
        ys, dy, w = (torch.randn(s, generator=g).to(dtype) for s in ((rows, d), (tokens, d), (tokens, k)))
        for weights in (w, None):
            w64 = None if weights is None else w.double()
            wc = None if weights is None else w.cuda()
            terms = combine64(ys.double(), place, w64)
            within(tk.combine(ys.cuda(), place.cuda(), wc), terms.sum(1), terms.abs().sum(1), k, dtype)
            dys, size, dw, dwsize = backward64(dy.double(), ys.double(), place, w64)
            got = tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), wc)
            if kind == "once":
                assert torch.equal(got[0].cpu(), dys.to(dtype))
            else:
                within(got[0], dys, size, n, dtype)
            within(got[1], dw, dwsize, d, dtype)
            one = [tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), wc, need=need) for need in ((True, False), (False, True), (False, False))]
            assert torch.equal(one[0][0], got[0]) and one[0][1] is None and torch.equal(one[1][1], got[1]) and one[1][0] is None
            assert one[2] == (None, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [1, 40, 257, 2100])
def test_rows_that_many_places_list(tk, d, dtype):
    """From none to some hundred places a row, on both sides of what a warp ranks; the sums are in the order of the places, so a call
    gives the same bits whenever it runs."""
    g = gen(d)
    times = [0, 1, 2, 3, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 1, 700, 2, 0, 1, 5]
    k = 4
    flat = torch.cat([torch.full((t,), r) for r, t in enumerate(times)] + [torch.tensor([-1, len(times), 1 << 40])])
    flat = torch.cat([flat, torch.full((-flat.numel() % k,), -1)])
    place = flat[torch.randperm(flat.numel(), generator=g)].view(-1, k)
    tokens, rows = place.shape[0], len(times)
    dy, ys, w = (torch.randn(s, generator=g).to(dtype) for s in ((tokens, d), (rows, d), (tokens, k)))
    for weights in (w, None):
        wc = None if weights is None else weights.cuda()
        dys, size, dw, dwsize = backward64(dy.double(), ys.double(), place, None if weights is None else weights.double())
        got = tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), wc)
        # a sum of m products: m roundings of its row
        m = torch.tensor(times, dtype=torch.float64)[:, None]
        assert bool(((got[0].double().cpu() - dys).abs() <= m * 2.0 ** -24 * size + half_step(dtype) * dys.abs() + 1e-38).all())
        within(got[1], dw, dwsize, d, dtype)
        on = dy.cuda(), ys.cuda(), place.cuda(), wc
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = tk.combine_backward(*on)
        for _ in range(5):
            again = tk.combine_backward(*on)
            graph.replay()
            assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(again, got, out))
    dy, w = torch.randint(-2, 3, (tokens, d), generator=g).to(dtype), torch.randint(0, 2, (tokens, k), generator=g).to(dtype)
    want = backward64(dy.double(), ys.double(), place, w.double())[0].to(dtype)
    assert torch.equal(tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), w.cuda())[0].cpu(), want)


def test_the_time_of_rows_listed_twice_grows_with_the_places(tk):
    """Eight times the places take about eight times as long, not sixty-four: a quarter of that is the border."""
    g = torch.Generator(device="cuda").manual_seed(11)
    took = []
    for tokens in (4096, 32768):
        place = torch.randperm(tokens * 8, device="cuda", generator=g).remainder_(tokens * 4).view(tokens, 8)
        dy, ys = torch.randn(tokens, 64, device="cuda", generator=g), torch.randn(tokens * 4, 64, device="cuda", generator=g)
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            tk.combine_backward(dy, ys, place, need=(True, False))
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
        dys = tk.combine_backward(dy, ys, place, need=(True, False))[0]
        order = place.view(-1).sort(stable=True).indices.view(-1, 2) // 8
        assert torch.equal(dys, dy[order[:, 0]] + dy[order[:, 1]])
    assert took[1] <= 16 * took[0], took


@pytest.mark.parametrize("dtype", DTYPES)
def test_whole_numbers_are_exact(tk, dtype):
    g = gen(3)
    tokens, k, rows, d = 600, 8, 900, 200
    place = torch.randint(-5, rows + 5, (tokens, k), generator=g)
    ys, dy, w = (torch.randint(-2, 3, s, generator=g).to(dtype) for s in ((rows, d), (tokens, d), (tokens, k)))
    assert torch.equal(tk.combine(ys.cuda(), place.cuda(), w.cuda()).cpu(), combine64(ys.double(), place, w.double()).sum(1).to(dtype))
    dys, _, dw, _ = backward64(dy.double(), ys.double(), place, w.double())
    got = tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), w.cuda())
    assert torch.equal(got[0].cpu(), dys.to(dtype)) and torch.equal(got[1].cpu(), dw.to(dtype))
    # one row for every place
    place[:] = 7
    dys, size, dw, _ = backward64(dy.double(), ys.double(), place, w.double())
    got = tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), w.cuda())
    assert torch.equal(got[0].cpu(), dys.to(dtype)) and torch.equal(got[1].cpu(), dw.to(dtype))


def test_strided_rows(tk):
    for dtype in DTYPES:
        g = gen(4)
        place = torch.randperm(400, generator=g).view(100, 4).cuda()
        w = torch.randn(100, 4, generator=g).to(dtype).cuda()
        by, bdy = torch.randn(400, 300, generator=g).to(dtype).cuda(), torch.randn(100, 300, generator=g).to(dtype).cuda()
        for o in (0, 8, 1):
            ys, dy = by[:, o:o + 256], bdy[:, o:o + 256]
            assert torch.equal(tk.combine(ys, place, w), tk.combine(ys.contiguous(), place, w))
            for a, b in zip(tk.combine_backward(dy, ys, place, w), tk.combine_backward(dy.contiguous(), ys.contiguous(), place, w)):
                assert (a.double() - b.double()).abs().max() <= 256 * 2.0 ** -16 * b.double().abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [256, 255, 1001])
def test_strided_rows_give_the_gradients_of_contiguous_ones(tk, dtype, d):
    """Rows that start on 16-byte boundaries and off them.  Each row of dys is one product, bit for bit; dweights' sums of d products
    may be formed in another order on the other path."""
    g = gen(d)
    place = torch.randperm(400, generator=g).view(100, 4)
    ys, dy, w = (torch.randn(s, generator=g).to(dtype) for s in ((400, d), (100, d), (100, 4)))
    want, _, dw, size = backward64(dy.double(), ys.double(), place, w.double())
    for o, gap in ((0, 8), (8, 48), (1, 0), (3, 5), (0, 1)):
        by, bdy = torch.full((400, o + d + gap), torch.nan, dtype=dtype, device="cuda"), torch.full((100, o + d + gap), torch.nan, dtype=dtype, device="cuda")
        by[:, o:o + d], bdy[:, o:o + d] = ys.cuda(), dy.cuda()
        got = tk.combine_backward(bdy[:, o:o + d], by[:, o:o + d], place.cuda(), w.cuda())
        assert torch.equal(got[0].cpu(), want.to(dtype))
        within(got[1], dw, size, d, dtype)
        y = combine64(ys.double(), place, w.double())
        within(tk.combine(by[:, o:o + d], place.cuda(), w.cuda()), y.sum(1), y.abs().sum(1), 4, dtype)


def test_values_that_are_not_finite_stay_in_their_rows(tk):
    g = gen(5)
    place = torch.randperm(300, generator=g).view(100, 3)
    place[9] = -1
    ys, w, dy = torch.randn(300, 64, generator=g), torch.rand(100, 3, generator=g), torch.randn(100, 64, generator=g)
    ys[int(place[5, 1])] = torch.inf
    ys[int(place[6, 2])] = torch.nan
    dy[9] = torch.nan        # (a dropped token's)
    y = tk.combine(ys.cuda(), place.cuda(), w.cuda())
    assert bool((y[5] == torch.inf).all()) and bool(y[6].isnan().all()) and bool((y[9] == 0).all())
    assert bool(y[[0, 1, 2, 3, 4, 7, 8]].isfinite().all())
    dys, dw = tk.combine_backward(dy.cuda(), ys.cuda(), place.cuda(), w.cuda())
    assert bool(dys.isfinite().all()) and bool((dw[9] == 0).all()) and bool(dw[10:].isfinite().all())


@pytest.mark.parametrize("dtype", [torch.float32])
def test_gradients_against_differences_and_autograd(tk, dtype):
    """A layer of experts: select, dispatch, one product an expert, combine, and back, against autograd in 64 bits."""
    g = gen(6)
    tokens, k, experts, d = 50, 2, 6, 32
    x, router, we = torch.randn(tokens, d, generator=g), torch.randn(experts, d, generator=g), torch.randn(experts, d, d, generator=g) / 6
    dy = torch.randn(tokens, d, generator=g)
    X, R, W = x.cuda(), router.cuda(), we.cuda()
    vals, idx = tk.select(tk.linear(X, R), k)
    weights = torch.softmax(vals, 1)
    xs, place, offsets = tk.dispatch(X, idx, experts)
    o = offsets.tolist()
    ys = torch.cat([tk.linear(xs[o[e]:o[e + 1]], W[e], act="silu") for e in range(experts)])
    pre = torch.cat([tk.linear(xs[o[e]:o[e + 1]], W[e]) for e in range(experts)])
    y = tk.combine(ys, place, weights)
    dys, dw = tk.combine_backward(dy.cuda(), ys, place, weights)
    dxs, dwe = torch.empty_like(xs), torch.zeros_like(W)
    for e in range(experts):
        s = slice(o[e], o[e + 1])
        dxs[s], dwe[e], _ = tk.linear_backward(dys[s], xs[s], W[e], pre=pre[s], act="silu")
    dx = tk.combine(dxs, place)

    def loss(x, w, we):
        z = torch.nn.functional.silu(torch.einsum("td,tkod->tko", x, we[idx.cpu()]))
        return ((z * w[..., None]).sum(1) * dy.double()).sum()

    a = [t.double().requires_grad_() for t in (x, weights.cpu(), we)]
    want = torch.autograd.grad(loss(*a), a)
    z = (torch.nn.functional.silu(torch.einsum("td,tkod->tko", a[0], a[2][idx.cpu()])) * a[1][..., None]).sum(1).detach()
    # sums of at most 64 products through two layers: 1e-4 of the largest is some hundred roundings
    for got, ref in ((y, z), (dx, want[0]), (dw, want[1]), (dwe, want[2])):
        assert float((got.double().cpu() - ref).abs().max()) <= 1e-4 * float(ref.abs().max())
    eps, u = 1e-5, torch.randn(tokens, k, generator=g).double()
    num = (loss(x.double(), weights.cpu().double() + eps * u, we.double()) - loss(x.double(), weights.cpu().double() - eps * u, we.double())) / (2 * eps)
    assert abs(float((dw.double().cpu() * u).sum() - num)) <= 1e-4 * float(dw.double().norm() * u.norm())


def test_capture_streams_and_no_tokens(tk):
    g = gen(7)
    a = [torch.randn(900, 128, generator=g).cuda(), routed(900, 4, 32, 8).cuda()]
    b = [torch.randn(900, 128, generator=g).cuda(), routed(900, 4, 32, 9).cuda()]
    w = torch.randn(900, 4, generator=g).cuda()

    def run(x, idx, stream=None):
        xs, place, offsets = tk.dispatch(x, idx, 32, stream=stream)
        y = tk.combine(xs, place, w, stream=stream)
        return [xs, place, offsets, y, *tk.combine_backward(y, xs, place, w, stream=stream)]

    want = run(*a), run(*b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(*a, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    graphs = []
    for _ in range(2):
        graph, s = torch.cuda.CUDAGraph(), [t.clone() for t in a]
        with torch.cuda.graph(graph):
            out = run(*s)
        graphs.append((graph, s, out))
    for new, ref in ((b, want[1]), (a, want[0])):
        for graph, s, out in graphs:
            s[0].copy_(new[0]), s[1].copy_(new[1])
            graph.replay()
        run(*b)
        torch.cuda.synchronize()
        for _, _, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, ref))
    xs, place, offsets = tk.dispatch(a[0][:0], a[1][:0], 32)
    assert xs.shape == (0, 128) and place.shape == (0, 4) and not offsets.any()
    dys, dw = tk.combine_backward(a[0][:0], want[0][0], place, w[:0])
    assert dw.shape == (0, 4) and dys.shape == want[0][0].shape and not dys.any()
    assert not tk.combine(want[0][0][:0], a[1], w).any()


def test_refusals(tk):
    x, idx = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for call, kind in ((lambda: tk.dispatch(x, idx.int(), 4), TypeError), (lambda: tk.dispatch(x, idx[:3], 4), ValueError),
                       (lambda: tk.dispatch(x, idx[:, :0], 4), ValueError), (lambda: tk.dispatch(x.half(), idx, 4), TypeError),
                       (lambda: tk.dispatch(x.t(), idx, 4), ValueError), (lambda: tk.dispatch(x, idx, 0), tk.TopkError),
                       (lambda: tk.dispatch(x, idx, 4097), tk.TopkError), (lambda: tk.combine(x, idx, x), ValueError),
                       (lambda: tk.combine(x, idx, idx), TypeError), (lambda: tk.combine(x[0], idx), ValueError),
                       (lambda: tk.combine_backward(x, x[:, :4], idx), ValueError), (lambda: tk.combine_backward(x[:3], x, idx), ValueError),
                       (lambda: tk.combine_backward(x, x.double(), idx), TypeError)):
        with pytest.raises(kind):
            call()


def test_need_that_is_neither_true_nor_false(tk):
    dy, ys, place = torch.ones(2, 8, device="cuda"), torch.ones(2, 8, device="cuda"), torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    for need in ((torch.ones(2), True), (True, torch.ones(2)), (True,)):
        with pytest.raises((RuntimeError, TypeError)):
            tk.combine_backward(dy, ys, place, need=need)
    dys, dw = tk.combine_backward(dy, ys, place, need=(0, 1))
    assert dys is None and torch.equal(dw, torch.full((2, 1), 8.0, device="cuda"))
