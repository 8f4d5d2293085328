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
