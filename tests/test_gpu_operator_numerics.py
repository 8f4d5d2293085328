"""The operators' arithmetic on the GPU where it could go wrong: long sums, values at the ends of f32's range, tails.

Every case is compared with 64-bit arithmetic on the CPU, within a bound that is derived beside it.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tk():
    import top_selection_prof_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normals(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def rounds_from(got, want, off):
    """Each value of got is the rounding (which is monotone) of some f32 value within `off` of want."""
    got = got.cpu()
    low, high = ((want + d).float().to(got.dtype) for d in (-off, off))
    bad = ~((got >= low) & (got <= high))
    assert not bad.any(), "%d of %d outside" % (int(bad.sum()), bad.numel())


@pytest.mark.parametrize("rows,inner,outer", [(64, 32768, 48), (300, 20000, 520), (600, 8200, 13000)])
def test_long_bf16_sums_stay_f32(tk, rows, inner, outer):
    """Sums of one sign, the residual taking nearly all of them away, so that what is left shows the f32 sum's error.

    The tensor cores cut a sum off after each 16 products: 128 cuts of at most 2^-23 of it in a round of 2048, then an f32
    rounding (2^-24) for each round and for each of at most 16 parts of k.
    """
    g = gen(inner)
    x, w = normals((rows, inner), torch.bfloat16, g).abs(), normals((outer, inner), torch.bfloat16, g).abs()
    s = (x.cuda().double() @ w.cuda().double().T).cpu()
    r = -s.bfloat16()
    y = tk.linear(x.cuda(), w.cuda(), residual=r.cuda())
    rounds_from(y, s + r.double(), (128 * 2.0 ** -23 + (inner / 2048 + 16) * 2.0 ** -24) * s)


def phi(z):
    return torch.exp(-0.5 * z * z) * 0.3989422804014327


def slope64(z, act):
    s = torch.sigmoid(z)
    return torch.special.ndtr(z) + z * phi(z) if act == "gelu" else s * (1 + z * (1 - s))


# rows, inner, outer: products on the tensor cores, by passes over few rows (dx of 5 and 24, dw of both), rows on and off
# 16-byte boundaries
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("rows,inner,outer", [(300, 96, 104), (257, 77, 99), (5, 96, 100), (24, 77, 99), (700, 260, 333)])
def test_smooth_bf16_gradients_keep_dz(tk, rows, inner, outer, act):
    """dz = dy act'(pre) has no bf16 value: rounding it to one before the products would show in every sum.

    dz enters with 16 bits (2^-17 of it) and its own f32 error (16 units of 2^-23 of |dy| (|slope| + 0.25)); a sum of n
    products in f32 is within n + 4 units of 2^-23 of the magnitudes.
    """
    g = gen(rows + outer)
    bf = torch.bfloat16
    x, w, dy = normals((rows, inner), bf, g), normals((outer, inner), bf, g), normals((rows, outer), bf, g)
    pre = normals((rows, outer), bf, g, 2.0)
    dx, dw, _ = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda(), pre=pre.cuda(), act=act)
    slope = slope64(pre.double(), act)
    dz, mag = dy.double() * slope, dy.double().abs() * (slope.abs() + 0.25)
    for got, want, m, n in ((dx, dz @ w.double(), mag @ w.double().abs(), outer),
                            (dw, dz.T @ x.double(), mag.T @ x.double().abs(), rows)):
        rounds_from(got, want, ((n + 4 + 16) * 2.0 ** -23 + 2.0 ** -17) * m)


@pytest.mark.parametrize("rows", [5, 30, 300])
def test_smooth_bf16_gradients_keep_infinities(tk, rows):
    """An infinity in w or x meets one sign of each dz, whatever parts dz enters in; dz of infinity and NaN likewise."""
    g = gen(rows)
    bf, inner, outer = torch.bfloat16, 96, 200
    x, w = normals((rows, inner), bf, g).abs() + 0.1, normals((outer, inner), bf, g).abs() + 0.1
    dy, pre = normals((rows, outer), bf, g).abs() + 0.1, normals((rows, outer), bf, g).abs() + 0.1
    x[2, 6], w[140, 95], w[3, 0] = torch.inf, -torch.inf, torch.inf
    for bad in (False, True):
        if bad:
            dy[1, 5], dy[4, 9] = torch.inf, torch.nan
        dz = dy.double() * slope64(pre.double(), "silu")
        dx, dw, _ = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda(), pre=pre.cuda(), act="silu")
        for got, want, n in ((dx, dz @ w.double(), outer), (dw, dz.T @ x.double(), rows)):
            same = want.isnan() | want.isinf()
            assert torch.equal(got.cpu().double()[same].nan_to_num(7.0), want[same].nan_to_num(7.0))
            # all terms positive; dz has bf16's own bits at least (2^-8 of it)
            want = torch.where(same, torch.zeros_like(want), want)
            rounds_from(torch.where(same, 0, got.cpu()), want, (2.0 ** -8 + (n + 20) * 2.0 ** -23) * want)


@pytest.mark.parametrize("inner", [1, 2])
def test_f32_products_of_parts_keep_all_bits(tk, inner):
    """Operands whose low bits are all ones, in sums so short that nothing else hides what a product of parts drops.

    Each of the inner products, and the sum, is cut off by at most 2^-23 of the result; the dropped products of parts are at
    most 2^-24 of a product, and the cuts of the smaller ones 6 x 2^-30.
    """
    g = gen(inner)
    top = torch.randint(0, 128, (200, 2), generator=g, dtype=torch.int32)
    sign = torch.randint(0, 2, (200, 1), generator=g, dtype=torch.int32)
    bits = (0x3F80FFFF + (top << 16)) | (sign << 31)
    x, w = bits[:100, :inner].contiguous().view(torch.float32), bits[100:, :inner].contiguous().view(torch.float32)
    x[0], w[0] = 1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -7 - 2.0 ** -23
    want = x.double() @ w.double().T
    got = tk.linear(x.cuda(), w.cuda()).double().cpu()
    assert float(((got - want) / want).abs().max()) <= (inner + 1 + 0.5 + 6 / 128) * 2.0 ** -23


def test_f32_products_at_the_end_of_the_range(tk):
    """Values whose leading bf16 part would be infinite; a product with them is finite all the same."""
    big = torch.tensor([[3.4028234e38], [3.3953139e38], [-3.4e38], [3.38e38]]).repeat(20, 1)
    w = torch.tensor([[0.5], [1.0], [2.0 ** -100], [0.0]]).repeat(20, 1)
    got = tk.linear(big.cuda(), w.cuda()).double().cpu()
    want = big.double() @ w.double().T
    assert float(((got - want).abs() / want.abs().clamp(min=1e-300)).max()) <= 2.0 ** -22


def spread(shape, g, low, high):
    """Values of either sign with random bits, their exponents uniform over [low, high]."""
    m = 1 + torch.rand(shape, generator=g, dtype=torch.float64)
    e = torch.randint(low, high + 1, shape, generator=g).double()
    return (torch.where(torch.rand(shape, generator=g) < 0.5, -m, m) * 2.0 ** e).float()


# exponents of x and of w: x near f32's smallest normal values, below them, over a wide range, both operands small, a small
# one that meets a large one (a product that no scaling holds), and ordinary ones
ENDS = [((-125, -112), (0, 0)), ((-147, -127), (1, 2)), ((-140, 5), (-3, 3)), ((-140, -20), (-140, 20)), ((-140, 40), (-140, 40)),
        ((-126, -100), (60, 126)), ((90, 100), (20, 22))]


@pytest.mark.parametrize("x_ends,w_ends", ENDS)
@pytest.mark.parametrize("rows,inner,outer", [(70, 3, 90), (300, 200, 264)])
def test_f32_products_over_the_whole_range(tk, rows, inner, outer, x_ends, w_ends):
    """Every value of f32 keeps its bits, and each row its own scale: the bound of an f32 sum, or of a denormal's spacing."""
    g = gen(rows + x_ends[0] + w_ends[0])
    x, w = spread((rows, inner), g, *x_ends), spread((outer, inner), g, *w_ends)
    x[1], x[2, 0], w[5] = 0.0, 1.5, 0.0
    b = spread((outer,), g, -130, -126)
    dy = spread((rows, outer), g, *x_ends)
    y = tk.linear(x.cuda(), w.cuda(), b.cuda())
    dx, dw, _ = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    x, w, b, dy = x.double(), w.double(), b.double(), dy.double()
    for got, p, q, more in ((y, x, w.T, b), (dx, dy, w, 0.0 * w[:1]), (dw, dy.T, x, 0.0 * x[:1])):
        want, mag, n = p @ q + more, p.abs() @ q.abs() + more.abs(), p.shape[1]
        got = got.double().cpu()
        end = want.abs() >= 2.0 ** 127
        bound = (n + 4) * 2.0 ** -23 * mag + n * 2.0 ** -149
        assert bool(((got - want).abs() <= bound)[~end].all()), float(((got - want).abs() / bound)[~end].max())


def test_small_and_infinite_values_together(tk):
    g = gen(3)
    x, w = spread((60, 40), g, -120, -115), spread((50, 40), g, 0, 1)
    x[7, 3] = torch.inf
    want = x.double() @ w.double().T
    got = tk.linear(x.cuda(), w.cuda()).double().cpu()
    assert torch.equal(got[7], want[7])
    rest = torch.arange(60) != 7
    bound = 44 * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)[rest]
    assert bool(((got - want).abs()[rest] <= bound).all())


def gelu_and_slope(z):
    below = 0.5 * torch.special.erfc(z * -0.5 ** 0.5)   # (ndtr cancels, in 64 bits too)
    return z * below, below + z * phi(z), below + z.abs() * phi(z)


def silu_and_slope(z):
    # (sigmoid(z) itself, not 1 - sigmoid(-z), so that nothing cancels)
    s = torch.exp(-torch.nn.functional.softplus(-z))
    t = torch.exp(-torch.nn.functional.softplus(z))
    return z * s, s * (1 + z * t), s * (1 + z.abs() * t)


def values_and_slopes(tk, z, act):
    """act(z) by few rows and by many, act'(z): each a value of z by itself."""
    one = torch.ones(2, 1, dtype=z.dtype, device="cuda")
    many = tk.linear(z.cuda()[:, None], one, act=act)[:, 0]
    few = torch.cat([tk.linear(p[:, None].contiguous(), one, act=act)[:, 1] for p in z.cuda().split(31)])
    dy, x = torch.ones(1, z.numel(), dtype=z.dtype, device="cuda"), torch.ones(1, 1, dtype=z.dtype, device="cuda")
    w = torch.ones(z.numel(), 1, dtype=z.dtype, device="cuda")
    slope = tk.linear_backward(dy, x, w, pre=z.cuda()[None], act=act, need=(False, False, True))[2]
    return many, few, slope


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gelu_in_its_tails(tk, dtype):
    """Within a few units of each value, not of the largest.

    f32: z^2 2^-23 from the rounding of the arguments of erfc and exp (whose logarithms change by z^2 / 2 times theirs), 4 units
    of 2^-23 for the functions and 4 for the operations; bf16: 4.8e-6 for the fitted tail and 2^-22 for each approximation.
    """
    z = torch.linspace(-9, 9, 2001).to(dtype)
    value, slope, mag = gelu_and_slope(z.double())
    rel = (z.double() ** 2 + 8) * 2.0 ** -23 + (4.8e-6 + 2.0 ** -20 if dtype == torch.bfloat16 else 0.0)
    many, few, got = values_and_slopes(tk, z, "gelu")
    rounds_from(many, value, rel * value.abs())
    rounds_from(few, value, rel * value.abs())
    rounds_from(got, slope, rel * mag)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_silu_in_its_tails(tk, dtype):
    """The same: 8 units of 2^-23 (bf16: 2^-20 for the approximations), z's exponential to its argument's rounding, and, where
    e^z is denormal, its spacing (bf16: the approximation has no denormal values, so 2^-126) times |z|."""
    z = torch.cat([torch.linspace(-103, 20, 3001), torch.linspace(-3, 3, 601)]).to(dtype)
    value, slope, mag = silu_and_slope(z.double())
    bf16 = dtype == torch.bfloat16
    rel = (z.double().abs() + 8) * 2.0 ** -23 + (2.0 ** -20 if bf16 else 0.0)
    end = (z.double().abs() + 2) * 2.0 ** (-126 if bf16 else -149)
    many, few, got = values_and_slopes(tk, z, "silu")
    rounds_from(many, value, rel * value.abs() + end)
    rounds_from(few, value, rel * value.abs() + end)
    rounds_from(got, slope, rel * mag + end)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [[20_000], [70_001], [1 << 22, 3, 100_003]])
@pytest.mark.parametrize("value", [0.7, 0.1, 0.3, 1.9, None])
def test_norm_of_equal_values(tk, value, sizes, dtype):
    """Roundings that all go one way: four f32 squares (eight of bf16, exact) in one f32 sum are within 2.5 (4.4) x 2^-24 of
    it, the sums of those lose 2^-47, the root halves that, and the norm's own rounding adds 2^-24."""
    g = gen(7)
    ts = [normals((n,), dtype, g) if value is None else torch.full((n,), value, dtype=dtype) for n in sizes]
    want = float(torch.cat(ts).double().norm())
    dev = [t.cuda() for t in ts]
    assert abs(float(tk.grad_norm(dev)) - want) <= (4.4 / 2 + 1) * 2.0 ** -24 * want
    assert abs(float(tk.clip_grad_norm_(dev, 1.0)) - want) <= (4.4 / 2 + 1) * 2.0 ** -24 * want
