"""The operators around the selection on the GPU against plain 64-bit forms on the CPU.

Two kinds of inputs.  Small integers: every product and every sum is a whole
number below 2^24, so f32 arithmetic is exact in any order and the result is
one rounding of the true value: outputs are compared bit for bit, and a lost,
doubled or misplaced term cannot hide.  Normal values: the bound on a sum of
n products formed in f32 in any order is n 2^-23 times the sum of their
magnitudes (products rounded or truncated, sums truncated: twice the 2^-24 of
rounding), to which the result's own rounding (2^-8 of it for bf16: one half
of the 2^-7 spacing, 2^-23 for f32) is added.
"""
import math

import numpy as np
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


def ints(shape, dtype, g, low=-2, high=2):
    return torch.randint(low, high + 1, shape, generator=g).to(dtype)


def normals(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def strided(t, extra=3, offset=1):
    """The same matrix on the GPU, its rows further apart and not on 16-byte boundaries."""
    big = torch.full((t.shape[0], t.shape[1] + extra), 7, dtype=t.dtype, device="cuda")
    v = big[:, offset:offset + t.shape[1]]
    v.copy_(t)
    return v


def half_spacing(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23


def same_bits(got, want64, what=""):
    want = want64.to(got.dtype)
    assert got.shape == want.shape, what
    got = got.cpu()
    assert torch.equal(got, want), "%s: %d values differ, first %s" % (what, int((got != want).sum()),
                                                                      (got != want).nonzero()[:1].tolist())


def within(got, want, magnitude, n, what=""):
    """|got - want| <= n 2^-23 magnitude + the rounding of the result."""
    got = got.double().cpu()
    bound = (n + 4) * 2.0 ** -23 * magnitude + half_spacing_of[0] * want.abs() + 1e-30
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d outside, worst %g of the bound" % (what, int(bad.sum()),
                                                                    float(((got - want).abs() / bound).max()))


half_spacing_of = [0.0]


@pytest.fixture(autouse=True)
def _spacing(request):
    dtype = request.node.callspec.params.get("dtype") if hasattr(request.node, "callspec") else None
    half_spacing_of[0] = half_spacing(dtype) if dtype is not None else half_spacing(torch.float32)


# ---- plain forms, 64 bits --------------------------------------------------------
def phi(z):
    return torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * torch.special.ndtr(z),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def slope64(z, act):
    s = torch.sigmoid(z)
    return {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(),
            "gelu": lambda: torch.special.ndtr(z) + z * phi(z), "silu": lambda: s * (1 + z * (1 - s))}[act]()


def dense(vals, idx, rows, n):
    """The selection as a dense matrix (places out of range left out, repeated ones added)."""
    d = torch.zeros(rows * n, dtype=torch.float64)
    flat = idx if idx.dim() == 1 else torch.where((idx >= 0) & (idx < n), idx + torch.arange(rows)[:, None] * n, -1)
    flat, v = flat.reshape(-1), vals.double().reshape(-1)
    ok = (flat >= 0) & (flat < rows * n)
    return d.index_add_(0, flat[ok], v[ok]).view(rows, n)


def at_places(full, idx):
    rows, n = full.shape
    if idx.dim() == 1:
        ok = (idx >= 0) & (idx < rows * n)
        return torch.where(ok, full.reshape(-1)[idx.clamp(0, rows * n - 1)], 0.0)
    ok = (idx >= 0) & (idx < n)
    return torch.where(ok, full.gather(1, idx.clamp(0, n - 1)), 0.0)


# ---- linear -----------------------------------------------------------------------
SIZES = [(1, 1, 1), (1, 64, 40), (2, 7, 300), (3, 5, 7), (5, 200, 1000), (16, 513, 129), (17, 129, 65), (64, 96, 640),
         (128, 64, 128), (129, 130, 257), (130, 1000, 136), (300, 512, 264), (513, 72, 1030), (1000, 40, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_linear_is_exact_on_whole_numbers(tk, dtype, rows, inner, outer):
    g = gen(rows * 7 + inner * 3 + outer)
    x, w = ints((rows, inner), dtype, g), ints((outer, inner), dtype, g)
    b, r = ints((outer,), dtype, g, -9, 9), ints((rows, outer), dtype, g, -9, 9)
    z = x.double() @ w.double().T
    xd, wd = x.cuda(), w.cuda()
    same_bits(tk.linear(xd, wd), z, "product")
    same_bits(tk.linear(xd, wd, b.cuda(), act="relu"), (z + b.double()).clamp(min=0), "relu")
    y, pre = tk.linear(xd, wd, b.cuda(), act="relu", residual=r.cuda(), save_pre=True)
    same_bits(pre, z + b.double(), "pre")
    same_bits(y, (z + b.double()).clamp(min=0) + r.double(), "residual")
    # rows apart and off 16-byte boundaries, the residual overwritten by the result
    rs = strided(r, 5, 2)
    out = tk.linear(strided(x), strided(w, 2, 1), b.cuda(), residual=rs, out=rs)
    assert out is rs
    same_bits(out, z + b.double() + r.double(), "strided")
    # aligned rows further apart
    same_bits(tk.linear(strided(x, 64, 0), strided(w, 32 if inner % 8 == 0 else 5, 0)), z, "apart")


# More tiles than the GPU takes at once, over short and long inner extents: whole waves and a rest that does not fill one,
# few tiles with many products each, and (short inner) columns of tiles that a pair of blocks goes down.
MANY = [(300, 200, 20000), (600, 512, 13000), (1030, 72, 9001), (300, 520, 20000), (2100, 600, 2600), (500, 20000, 300),
        (40, 9000, 700)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", MANY)
def test_linear_over_many_tiles_is_exact_on_whole_numbers(tk, dtype, rows, inner, outer):
    g = gen(inner)
    x, w = ints((rows, inner), dtype, g), ints((outer, inner), dtype, g)
    b, r, dy = ints((outer,), dtype, g, -9, 9), ints((rows, outer), dtype, g, -9, 9), ints((rows, outer), dtype, g)
    xd, wd, bd, rd, dyd = (t.cuda() for t in (x, w, b, r, dy))
    z = (xd.double() @ wd.double().T + bd.double()).cpu()
    same_bits(tk.linear(xd, wd, bd, act="relu"), z.clamp(min=0), "relu")
    y, pre = tk.linear(xd, wd, bd, act="relu", residual=rd, save_pre=True)
    same_bits(pre, z, "pre")
    same_bits(y, z.clamp(min=0) + r.double(), "residual")
    same_bits(tk.linear(strided(x), strided(w, 1, 0), bd), z, "strided")
    dx, dw, db = tk.linear_backward(dyd, xd, wd)
    same_bits(dx, (dyd.double() @ wd.double()).cpu(), "dx")
    same_bits(dw, (dyd.double().T @ xd.double()).cpu(), "dw")
    same_bits(db, dy.double().sum(0), "dbias")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", [(1, 512, 300), (7, 33, 129), (150, 700, 260)])
def test_linear_on_normal_values(tk, dtype, rows, inner, outer, act):
    g = gen(inner)
    x, w = normals((rows, inner), dtype, g), normals((outer, inner), dtype, g, 2 * inner ** -0.5)
    b, r = normals((outer,), dtype, g), normals((rows, outer), dtype, g)
    z = x.double() @ w.double().T + b.double()
    mag = x.double().abs() @ w.double().abs().T + b.double().abs()
    # |act'| <= 1.13; the activation itself is formed in f32 (its own error: a few units of 2^-23 of |z| + 1)
    want = act64(z, act) + r.double()
    got = tk.linear(x.cuda(), w.cuda(), b.cuda(), act=act, residual=r.cuda())
    within(got, want, 1.13 * mag + 4 * (z.abs() + 1) + r.double().abs(), inner, act)


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_keeps_nan_and_infinity_in_their_rows_and_columns(tk, dtype):
    g = gen(1)
    for rows in (3, 140):
        x, w = normals((rows, 70), dtype, g).abs() + 0.1, normals((150, 70), dtype, g).abs() + 0.1
        x[1, 5], x[2, 6], w[140, 69] = math.nan, math.inf, math.inf
        want = x.double() @ w.double().T
        got = tk.linear(x.cuda(), w.cuda()).double().cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.isinf(), want.isinf())
        extremes = torch.tensor([[-math.inf], [math.inf], [-200.0], [200.0], [math.nan]], dtype=dtype)
        one = torch.ones((3, 1), dtype=dtype)
        for act in ("relu", "gelu", "silu"):
            y = tk.linear(extremes.cuda(), one.cuda(), act=act).float().cpu()
            assert torch.equal(y[:4], torch.tensor([0.0, math.inf, 0.0, 200.0])[:, None].expand(4, 3)), act
            assert y[4].isnan().all()


def test_linear_of_no_rows(tk):
    y = tk.linear(torch.empty(0, 8, device="cuda"), torch.ones(4, 8, device="cuda"))
    assert y.shape == (0, 4)
    dx, dw, db = tk.linear_backward(y, torch.empty(0, 8, device="cuda"), torch.ones(4, 8, device="cuda"))
    assert dx.shape == (0, 8) and not dw.any() and not db.any() and dw.shape == (4, 8) and db.shape == (4,)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_linear_backward_is_exact_on_whole_numbers(tk, dtype, rows, inner, outer):
    g = gen(rows * 11 + inner + outer)
    x, w, dy = ints((rows, inner), dtype, g), ints((outer, inner), dtype, g), ints((rows, outer), dtype, g)
    pre = ints((rows, outer), dtype, g, -1, 1)
    for act, place in (("none", lambda t: t.cuda()), ("relu", lambda t: t.cuda()), ("relu", strided),
                       ("none", lambda t: strided(t, 16, 8))):
        dz = dy.double() * slope64(pre.double(), act)
        dx, dw, db = tk.linear_backward(place(dy), place(x), place(w), pre=place(pre), act=act)
        same_bits(dx, dz @ w.double(), act + " dx")
        same_bits(dw, dz.T @ x.double(), act + " dw")
        same_bits(db, dz.sum(0), act + " dbias")
    only = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda(), need=(False, True, False))
    assert only[0] is None and only[2] is None
    same_bits(only[1], dy.double().T @ x.double(), "dw alone")
    only = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda(), pre=pre.cuda(), act="relu", need=(False, False, True))
    same_bits(only[2], (dy.double() * (pre.double() > 0)).sum(0), "dbias alone")


# Few rows: sums over outer in several chunks, rows past a group of eight, columns past a tile, aligned rows and others.
FEW = [(1, 512, 3000), (4, 1032, 700), (5, 515, 4001), (8, 300, 129), (9, 128, 65), (13, 261, 5000), (24, 130, 2100),
       (32, 516, 1000), (32, 77, 20011), (33, 77, 300), (48, 515, 900), (49, 515, 900)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", FEW)
def test_linear_backward_of_few_rows_is_exact_on_whole_numbers(tk, dtype, rows, inner, outer):
    g = gen(rows + inner * 5 + outer)
    x, w, dy = ints((rows, inner), dtype, g), ints((outer, inner), dtype, g), ints((rows, outer), dtype, g)
    for place in (lambda t: t.cuda(), strided, lambda t: strided(t, 16, 8)):
        dx, dw, db = tk.linear_backward(place(dy), place(x), place(w))
        same_bits(dx, dy.double() @ w.double(), "dx")
        same_bits(dw, dy.double().T @ x.double(), "dw")
        same_bits(db, dy.double().sum(0), "dbias")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", FEW + [(2, 2050, 33), (40, 515, 13000), (41, 515, 1300), (7, 9000, 33)])
def test_linear_of_few_rows_is_exact_on_whole_numbers(tk, dtype, rows, inner, outer):
    g = gen(rows + inner + outer)
    x, w, b = ints((rows, inner), dtype, g), ints((outer, inner), dtype, g), ints((outer,), dtype, g, -9, 9)
    z = x.double() @ w.double().T + b.double()
    for place in (lambda t: t.cuda(), strided, lambda t: strided(t, 16, 8)):
        same_bits(tk.linear(place(x), place(w), b.cuda(), act="relu"), z.clamp(min=0), "relu")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,inner,outer", [(3, 70, 150), (12, 515, 900), (31, 132, 2050)])
def test_linear_backward_of_few_rows_on_normal_values(tk, dtype, rows, inner, outer):
    g = gen(rows)
    x, w, dy = normals((rows, inner), dtype, g), normals((outer, inner), dtype, g, 0.1), normals((rows, outer), dtype, g)
    dx, dw, _ = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    x, w, dy = x.double(), w.double(), dy.double()
    within(dx, dy @ w, dy.abs() @ w.abs(), outer, "dx")
    within(dw, dy.T @ x, dy.abs().T @ x.abs(), rows, "dw")


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_backward_of_few_rows_keeps_nan_and_infinity_in_their_places(tk, dtype):
    g = gen(2)
    x, w, dy = (normals(s, dtype, g).abs() + 0.1 for s in ((5, 67), (301, 67), (5, 301)))
    dy[1, 5], x[2, 6], w[300, 66] = math.nan, math.inf, math.inf
    dx, dw, _ = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    for got, want in ((dx, dy.double() @ w.double()), (dw, dy.double().T @ x.double())):
        assert torch.equal(got.cpu().isnan(), want.isnan()) and torch.equal(got.cpu().isinf(), want.isinf())


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_backward_of_smooth_activations(tk, dtype, act):
    g = gen(5)
    rows, inner, outer = 67, 90, 301
    x, w, dy = normals((rows, inner), dtype, g), normals((outer, inner), dtype, g, 0.1), normals((rows, outer), dtype, g)
    pre = normals((rows, outer), dtype, g, 3.0)
    pre[0, :4] = torch.tensor([-math.inf, math.inf, -90.0, 90.0], dtype=dtype)
    slope = slope64(pre.double(), act)
    slope[0, 0], slope[0, 1] = 0.0, 1.0
    dz = dy.double() * slope
    # dz is rounded once (bf16) before the products, and the slope has a few f32 units of its own
    off = half_spacing(dtype) + 16 * 2.0 ** -23
    mag = dy.double().abs() * (slope.abs() + 0.25)
    dx, dw, db = tk.linear_backward(dy.cuda(), x.cuda(), w.cuda(), pre=pre.cuda(), act=act)
    for got, want, m, n in ((dx, dz @ w.double(), mag @ w.double().abs(), outer),
                            (dw, dz.T @ x.double(), mag.T @ x.double().abs(), rows)):
        within(got, want, m + (off * m) * 2.0 ** 23 / (n + 4), n, act)
    within(db, dz.sum(0), 16 * mag.sum(0), rows, act + " dbias")


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_gradients_against_differences(tk, act):
    """d/dt of sum(dy * linear(x + t u, w + t v, b + t c)) at 0, by central differences of the f32 forward."""
    g = gen(9)
    rows, inner, outer, h = 20, 48, 70, 2.0 ** -5
    x, w, b = (normals(s, torch.float32, g, f) for s, f in (((rows, inner), 1), ((outer, inner), 0.2), ((outer,), 1)))
    u, v, c = (normals(s, torch.float32, g, f) for s, f in (((rows, inner), 1), ((outer, inner), 0.2), ((outer,), 1)))
    dy = normals((rows, outer), torch.float32, g)

    def loss(t):
        args = [(p + t * q).float() for p, q in ((x, u), (w, v), (b, c))]
        return float((dy.double() * tk.linear(args[0].cuda(), args[1].cuda(), args[2].cuda(), act=act).double().cpu()).sum())

    y, pre = tk.linear(x.cuda(), w.cuda(), b.cuda(), act=act, save_pre=True)
    dx, dw, db = (t.double().cpu() for t in tk.linear_backward(dy.cuda(), x.cuda(), w.cuda(), pre=pre, act=act))
    slope = float((dx * u.double()).sum() + (dw * v.double()).sum() + (db * c.double()).sum())
    # z(t) = z + t p + t^2 q.  The third derivative of act(z(t)) is act''' p^3 + 6 act'' p q (|act'''| <= 0.8, |act''| <= 0.8)
    # plus terms in t; p is taken at its largest over the interval.  Rounding: inner 2^-23 of the magnitudes, over h.
    x, w, b, u, v, c = (t.double() for t in (x, w, b, u, v, c))
    q = (u @ v.T).abs()
    p = (x @ v.T + u @ w.T + c).abs() + 2 * h * q
    third = 0.8 * p ** 3 + 6 * 0.8 * p * q
    mag = (x.abs() + h * u.abs()) @ (w.abs() + h * v.abs()).T + b.abs() + h * c.abs()
    tol = float((dy.double().abs() * (h * h / 6 * (third if act != "none" else 0 * third) + 1.13 * (inner + 8) * 2.0 ** -23 * mag / h)).sum())
    assert abs((loss(h) - loss(-h)) / (2 * h) - slope) <= tol


# ---- selections -----------------------------------------------------------------
def flat_places(rows, n, count, g, skew=1.0):
    r = torch.randint(0, rows, (count,), generator=g)
    c = (n * torch.rand(count, generator=g, dtype=torch.float64) ** skew).long().clamp(max=n - 1)
    return r * n + c


# rows, n, d, count (flat), skew: groups of no, one, some (<= 64) and many (> 64, in pieces) places
FLAT = [(1, 1, 1, 1, 1), (1, 9, 3, 0, 1), (4, 10, 8, 3, 1), (5, 7, 33, 400, 1), (33, 50, 64, 500, 2), (64, 300, 129, 2000, 4),
        (100, 1000, 512, 3000, 3), (3, 2000, 257, 5000, 1), (700, 3, 72, 4000, 1), (50, 80, 1032, 900, 2),
        (9, 400, 2050, 300, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,d,count,skew", FLAT)
def test_flat_selection_is_exact_on_whole_numbers(tk, dtype, rows, n, d, count, skew):
    g = gen(rows + n + d + count)
    idx = flat_places(rows, n, count, g, skew)
    if count > 10:   # places out of range hold none; others are listed twice
        idx[3], idx[7], idx[8], idx[9] = -1, rows * n, -(1 << 40), 1 << 50
        idx[5] = idx[6]
    check_selection(tk, dtype, g, idx, rows, n, d)


# rows, n, d, k: k of one, up to one piece (64) and several
PER_ROW = [(1, 1, 1, 1), (1, 12288, 512, 64), (3, 100, 40, 65), (40, 64, 129, 7), (2, 3000, 520, 1000), (130, 20, 8, 20),
           (6, 30, 16, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,d,k", PER_ROW)
def test_per_row_selection_is_exact_on_whole_numbers(tk, dtype, rows, n, d, k):
    g = gen(rows + n + d + k)
    idx = torch.rand(rows, n, generator=g).argsort(1)[:, :k].contiguous()
    if k > 5:
        idx[0, 2], idx[-1, 4], idx[0, 1] = -1, n, 1 << 33
    check_selection(tk, dtype, g, idx, rows, n, d)


def check_selection(tk, dtype, g, idx, rows, n, d):
    vals, w, x, bias = ints(idx.shape, dtype, g), ints((n, d), dtype, g), ints((rows, d), dtype, g), ints((d,), dtype, g, -9, 9)
    dvals = ints(idx.shape, dtype, g)
    s, w64, x64 = dense(vals, idx, rows, n), w.double(), x.double()
    assert s.abs().sum(1).max() * 2 < 2 ** 24 and s.abs().sum(0).max() * 2 < 2 ** 24
    iv, vv, dv = idx.cuda(), vals.cuda(), dvals.cuda()
    for place in (lambda t: t.cuda(), strided, lambda t: strided(t, 24, 8)):
        wd, xd = place(w), place(x)
        same_bits(tk.decode(vv, iv, wd, rows, bias=bias.cuda()), s @ w64 + bias.double(), "decode")
        same_bits(tk.decode(vv, iv, wd, rows), s @ w64, "decode without bias")
        got = tk.decode_backward(xd, vv, iv, wd)
        same_bits(got[0], at_places(x64 @ w64.T, idx), "dvals")
        same_bits(got[1], s.T @ x64, "dw")
        same_bits(got[2], x64.sum(0), "dbias")
        same_bits(tk.decode_backward(xd, vv, iv, wd, need=(True, False, False))[0], got[0].double().cpu(), "dvals alone")
        same_bits(tk.decode_backward(xd, vv, iv, wd, need=(False, True, False))[1], got[1].double().cpu(), "dw alone")
        for act in ("relu", "none"):
            z = dense(torch.where(vals > 0, dvals, torch.zeros_like(dvals)) if act == "relu" else dvals, idx, rows, n)
            got = tk.linear_backward_selected(dv, vv, iv, xd, wd, act=act)
            same_bits(got[0], z @ w64, act + " dx")
            same_bits(got[1], z.T @ x64, act + " dw")
            same_bits(got[2], z.sum(0), act + " dbias")


@pytest.mark.parametrize("dtype", DTYPES)
def test_selection_on_normal_values_and_run_twice(tk, dtype):
    """Within the bound of 64 bits, and the same bits each time (no order of blocks or atomics in the results)."""
    g = gen(3)
    rows, n, d, count = 90, 500, 200, 6000
    idx = torch.randperm(rows * n, generator=g)[:count]
    idx[:3000] = torch.unique(flat_places(rows, n, 20000, g, 8.0))[:3000][torch.randperm(3000, generator=g)]
    vals, w, x = normals(idx.shape, dtype, g), normals((n, d), dtype, g), normals((rows, d), dtype, g)
    s, w64, x64 = dense(vals, idx, rows, n), w.double(), x.double()
    a64 = dense(vals.abs(), idx, rows, n)
    args = [t.cuda() for t in (vals, idx, w)]
    first = (tk.decode(*args, rows), *tk.decode_backward(x.cuda(), *args),
             *tk.linear_backward_selected(args[0], args[0], args[1], x.cuda(), args[2]))
    within(first[0], s @ w64, a64 @ w64.abs(), n)
    within(first[1], at_places(x64 @ w64.T, idx), at_places(x64.abs() @ w64.abs().T, idx), d)
    within(first[2], s.T @ x64, a64.T @ x64.abs(), rows)
    within(first[3], x64.sum(0), x64.abs().sum(0), rows)
    for _ in range(3):
        again = (tk.decode(*args, rows), *tk.decode_backward(x.cuda(), *args),
                 *tk.linear_backward_selected(args[0], args[0], args[1], x.cuda(), args[2]))
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_more_places_than_one_bitmap(tk):
    """A column with places past the 2^20th of the selection: its order spans several bitmaps."""
    g = gen(4)
    rows, n, d, count = 2000, 1000, 4, 1_300_000
    idx = torch.randperm(rows * n, generator=g)[:count]
    vals, x = normals((count,), torch.float32, g), normals((rows, d), torch.float32, g)
    w = normals((n, d), torch.float32, g)
    y = tk.decode(vals.cuda(), idx.cuda(), w.cuda(), rows)
    dvals, dw, _ = tk.decode_backward(x.cuda(), vals.cuda(), idx.cuda(), w.cuda())
    s, a = dense(vals, idx, rows, n), dense(vals.abs(), idx, rows, n)
    within(y, s @ w.double(), a @ w.double().abs(), n)
    within(dw, s.T @ x.double(), a.T @ x.double().abs(), rows)
    for _ in range(2):
        assert torch.equal(y, tk.decode(vals.cuda(), idx.cuda(), w.cuda(), rows))
        assert torch.equal(dw, tk.decode_backward(x.cuda(), vals.cuda(), idx.cuda(), w.cuda())[1])


def test_decode_gradients_against_differences(tk):
    """decode is linear in the values and in the dictionary: on whole numbers a unit step shows the gradient exactly."""
    g = gen(8)
    rows, n, d, count = 6, 40, 24, 60
    idx = torch.randperm(rows * n, generator=g)[:count]
    vals, w, dy = ints((count,), torch.float32, g), ints((n, d), torch.float32, g), ints((rows, d), torch.float32, g)

    def loss(v, m):
        return (dy.double() * tk.decode(v.cuda(), idx.cuda(), m.cuda(), rows).double().cpu()).sum()

    dvals, dw, _ = (t.cpu() for t in tk.decode_backward(dy.cuda(), vals.cuda(), idx.cuda(), w.cuda()))
    for s in (0, 11, 59):
        step = vals.clone()
        step[s] += 1
        assert float(loss(step, w) - loss(vals, w)) == float(dvals[s])
    for c, j in ((int(idx[0] % n), 0), (int(idx[11] % n), 23), (5, 5)):
        step = w.clone()
        step[c, j] += 1
        assert float(loss(vals, step) - loss(vals, w)) == float(dw[c, j])


def test_relaxed_recall_padding_decodes_to_nothing(tk):
    """Places that a selection did not fill (index -1, value -inf) add nothing."""
    w = torch.ones(5, 16, device="cuda")
    vals = torch.tensor([[2.0, -math.inf], [-math.inf, -math.inf]], device="cuda")
    idx = torch.tensor([[3, -1], [-1, -1]], device="cuda")
    y = tk.decode(vals, idx, w, 2)
    assert torch.equal(y.cpu(), torch.tensor([2.0, 0.0])[:, None].expand(2, 16))
    dv, dw, _ = tk.decode_backward(y, vals, idx, w)
    assert torch.equal(dv.cpu(), torch.tensor([[32.0, 0.0], [0.0, 0.0]]))
    assert torch.equal(dw.cpu(), torch.zeros(5, 16).index_fill_(0, torch.tensor([3]), 4.0))


# ---- gradient norm --------------------------------------------------------------
def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def clipped(t, norm32, max_norm):
    """The f32 formula: scale and product rounded once each, then the result to the tensor's type."""
    f = np.float32(max_norm) / (np.float32(norm32) + np.float32(1e-6))
    f = np.float32(min(f, np.float32(1.0)))
    return (t.float() * float(f)).to(t.dtype)


SIZE_LISTS = [[1], [7, 0, 8191, 8192, 8193], [100_003], [3] * 700, [1 << 20, 5, 77], [0, 0]]


@pytest.mark.parametrize("sizes", SIZE_LISTS, ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("share", [0.25, 1.5])
def test_clip_grad_norm(tk, sizes, share):
    g = gen(sum(sizes))
    # dtypes alternate; every third tensor starts off a 16-byte boundary
    host = [normals((n,), DTYPES[i % 2], g, 0.1) for i, n in enumerate(sizes)]
    dev = []
    for i, t in enumerate(host):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = buf[i % 3:i % 3 + t.numel()]
        v.copy_(t)
        dev.append(v)
    want = norm64(host)
    max_norm = share * want
    outs = [torch.full_like(t, 5.0) for t in dev]
    norm = tk.clip_grad_norm(dev, max_norm, out=outs)
    # squares and sums: at most 8 f32 roundings of relative size 2^-24 a value before f64 takes over, then one
    assert abs(float(norm) - want) <= 40 * 2.0 ** -24 * want
    assert float(tk.grad_norm(dev)) == float(norm)
    for t, o, d in zip(host, outs, dev):
        assert torch.equal(o.cpu(), clipped(t, float(norm), max_norm))
        assert torch.equal(d.cpu(), t)
    again = tk.clip_grad_norm_(dev, max_norm)
    assert float(again) == float(norm)
    for o, d in zip(outs, dev):
        assert torch.equal(o, d)


@pytest.mark.parametrize("scale", [1e30, 1e-25, 3e-38])
def test_norm_of_values_whose_squares_leave_f32(tk, scale):
    t = normals((5000,), torch.float32, gen(2)) * scale
    got = float(tk.grad_norm([t.cuda(), torch.zeros(3, device="cuda")]))
    assert abs(got - norm64([t])) <= 2.0 ** -23 * norm64([t])


def test_norm_that_is_not_finite(tk):
    t = torch.ones(100, device="cuda")
    t[5] = math.inf
    norm = tk.clip_grad_norm_([t], 1.0)
    assert math.isinf(float(norm)) and float(t[0]) == 0.0 and bool(t[5].isnan())
    t = torch.ones(100, device="cuda")
    t[7] = math.nan
    assert math.isnan(float(tk.clip_grad_norm_([t], 1.0))) and bool(t.isnan().all())
    t = torch.ones(64, device="cuda")
    assert float(tk.clip_grad_norm_([t], math.inf)) == 8.0 and bool((t == 1).all())
    assert float(tk.clip_grad_norm_([t], 0.0)) == 8.0 and not t.any()


# ---- as a user has them ------------------------------------------------------------
def test_another_stream_and_selections_in_between(tk):
    """The operators' scratch and the selection's do not meet; a side stream gives the same results."""
    g = gen(12)
    x, w = normals((300, 64), torch.bfloat16, g).cuda(), normals((4096, 64), torch.bfloat16, g, 0.125).cuda()
    b = normals((4096,), torch.bfloat16, g, 0.1).cuda()

    def step(stream=None):
        a = tk.linear(x, w, b, act="relu", stream=stream)
        v, i = tk.select_global(a, 9600, stream=stream)
        y = tk.decode(v, i, w, 300, stream=stream)
        dv, dw, db = tk.decode_backward(y, v, i, w, stream=stream)
        dx, dwe, dbe = tk.linear_backward_selected(dv, v, i, x, w, stream=stream)
        n = tk.clip_grad_norm_([dw, db, dwe, dbe], 1.0, stream=stream)
        return a, v, i, y, dv, dw, db, dx, dwe, dbe, n

    first = step()
    again = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    third = step(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for p, q, r, s in zip(first, again, other, third):
        assert torch.equal(p, q) and torch.equal(p, r) and torch.equal(p, s)


def test_autoencoder_step_against_autograd(tk):
    """The example's step: its gradients against torch's own through the same selection in 64 bits."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "batchtopk_autoencoder.py")
    spec = importlib.util.spec_from_file_location("batchtopk_autoencoder", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    rows, width, features, k = 96, 64, 700, 8
    model = ex.Autoencoder(width, features, k, dtype=torch.float32)
    data = ex.batches(width, 150, 6, rows, dtype=torch.float32)
    x = next(data)
    loss, y, grads = model.gradients(x)
    p = {n: t.double().cpu().requires_grad_() for n, t in model.params.items()}
    x64 = x.double().cpu()
    z = torch.relu(x64 @ p["w_enc"].T + p["b_enc"])
    top = z.detach().flatten().topk(rows * k + 1).values
    assert float(top[-2] - top[-1]) > 1e-6          # the f32 activations select the same places
    code = torch.where(z >= top[-2], z, 0.0)
    want_y = code @ p["w_dec"] + p["b_dec"]
    want = (want_y - x64).square().sum() / rows
    want.backward()
    # sums of at most max(rows, features, width) products, each factor itself such a sum: 4 n 2^-23 of the largest value's scale
    tol = 4 * features * 2.0 ** -23
    want, want_y = want.detach(), want_y.detach()
    assert abs(float(loss) - float(want)) <= tol * float(want)
    assert float((y.double().cpu() - want_y).abs().max()) <= tol * float(want_y.abs().max() + 1)
    for n, g in grads.items():
        scale = float(p[n].grad.abs().max())
        assert float((g.double().cpu() - p[n].grad).abs().max()) <= tol * max(scale, 1.0), n
    norm = float(model.step(x)[1])                  # the step itself: the norm of these gradients, and finite parameters
    whole = math.sqrt(sum(float(t.grad.square().sum()) for t in p.values()))
    assert abs(norm - whole) <= tol * whole
    assert all(bool(t.isfinite().all()) for t in model.params.values())


def test_refusals(tk):
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(6, 8, device="cuda")
    i, v = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.ones(3, device="cuda")
    for call in (lambda: tk.linear(x.cpu(), w), lambda: tk.linear(x, w.bfloat16()), lambda: tk.linear(x.double(), w.double()),
                 lambda: tk.linear(x, w, bias=v.bfloat16()), lambda: tk.decode(v, i.int(), w, 4),
                 lambda: tk.decode(v.bfloat16(), i, w, 4), lambda: tk.decode(v, i.cpu(), w, 4),
                 lambda: tk.grad_norm([x, x.cpu()]), lambda: tk.grad_norm([x.half()])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: tk.linear(x[0], w), lambda: tk.linear(x, w[:, :7]), lambda: tk.linear(x.T, w),
                 lambda: tk.linear(x, w, bias=v), lambda: tk.linear(x, w, act="tanh"), lambda: tk.linear(x, w, residual=x),
                 lambda: tk.linear(x[:1].expand(4, 8), w), lambda: tk.linear(x, w, out=x),
                 lambda: tk.linear_backward(torch.ones(4, 6, device="cuda"), x, w, act="relu"),
                 lambda: tk.linear_backward(x, x, w), lambda: tk.decode(v, i[:2], w, 4),
                 lambda: tk.decode(v[:, None], i[:, None], w, 4), lambda: tk.decode(v, i, w, 4, bias=v),
                 lambda: tk.decode_backward(x[:, :7], v, i, w), lambda: tk.grad_norm([]),
                 lambda: tk.clip_grad_norm([x], 1.0, out=[]), lambda: tk.clip_grad_norm([x], 1.0, out=[w]),
                 lambda: tk.grad_norm([x.T])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tk.linear_backward_selected(v, v, i, x, w, act="gelu"), lambda: tk.clip_grad_norm_([x], -1.0),
                 lambda: tk.clip_grad_norm_([x], math.nan), lambda: tk.linear(x[:, :0], w[:, :0])):
        with pytest.raises(tk.TopkError) as err:
            call()
        assert err.value.status == -1
    torch.cuda.synchronize()
