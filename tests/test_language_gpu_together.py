"""A small model's decoding loop out of the framework's operators, every call checked on its own inputs in 64 bits: a router's
selection, tokens to their experts and back, attention over a cache that is full and gives up a slot a step, the next token; and
the cache cut down at the end."""
import pytest
import torch

from .test_language_gpu_cache import evict64, replace64
from .test_language_gpu_experts import combine64, sort64
from .test_language_gpu_tokens import check, f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decoding_loop(dtype):
    import top_selection_prof_gb300 as tk
    g = torch.Generator().manual_seed(0)
    batch, d, experts, k, heads, dim, slots, vocabulary, steps = 3, 64, 8, 2, 2, 32, 16, 5003, 40

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()

    embed, router, head = normal(vocabulary, d), normal(experts, d, scale=d ** -0.5), normal(vocabulary, d, scale=0.3)
    we, wq, wk, wv = normal(experts, d, d, scale=d ** -0.5), normal(2 * heads * dim, d, scale=0.2), normal(heads * dim, d, scale=0.2), normal(heads * dim, d, scale=0.2)
    keys, values = torch.zeros(batch, heads, slots, dim, dtype=dtype, device="cuda"), torch.zeros(batch, heads, slots, dim, dtype=dtype, device="cuda")
    score, positions = torch.zeros(batch, heads, slots, device="cuda"), torch.zeros(batch, heads, slots, dtype=torch.int64, device="cuda")
    weights = None
    tokens = torch.tensor([1, 2, 3], device="cuda")
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    seen_tokens = set()
    for step in range(steps):
        x = embed[tokens]
        vals, idx = tk.select(tk.linear(x, router), k)
        mix = torch.softmax(vals.float(), 1).to(dtype)
        xs, place, offsets = tk.dispatch(x, idx, experts)
        p, o, order = sort64(idx.cpu(), experts)
        assert torch.equal(place.cpu(), p) and torch.equal(offsets.cpu(), o) and torch.equal(xs.cpu(), x.cpu()[order // k])
        at = offsets.tolist()
        ys = torch.cat([tk.linear(xs[at[e]:at[e + 1]], we[e], act="silu") for e in range(experts)])
        y = tk.combine(ys, place, mix)
        terms = combine64(ys.cpu().double(), place.cpu(), mix.cpu().double())
        assert bool(((y.cpu().double() - terms.sum(1)).abs() <= k * 2.0 ** -24 * terms.abs().sum(1) + half * terms.sum(1).abs() + 1e-30).all())
        q, nk, nv = (tk.linear(y, w).view(batch, -1, dim) for w in (wq, wk, wv))
        lengths = torch.full((batch,), step, device="cuda")
        state = dict(keys=keys, values=values, score=score, positions=positions, lengths=lengths, key=nk, value=nv, weights=weights)
        want, want_slots = replace64({n: None if t is None else t.cpu().clone() for n, t in state.items()}, 4)
        got = tk.replace_(keys, values, score, positions, lengths, nk, nv, recent=4, weights=weights)
        assert torch.equal(got.cpu(), want_slots)
        for n in ("keys", "values", "positions"):
            assert torch.equal(state[n].cpu(), want[n]), n
        # (sums of three f32 weights in 64 bits and in pairs of f32: the same rounding but for 2^-44 of them)
        assert bool(((score.cpu().double() - want["score"].double()).abs() <= 2.0 ** -23 * want["score"].double().abs()).all())
        # attention of this step's query, in torch: two query heads a head
        a = torch.einsum("bhgd,bhsd->bhgs", q.view(batch, heads, 2, dim).float(), keys.float()) * dim ** -0.5
        a = a.masked_fill(torch.arange(slots, device="cuda") > step, -torch.inf).softmax(-1)
        weights = a.reshape(batch, 2 * heads, 1, slots).contiguous()
        out = torch.einsum("bhgs,bhsd->bhgd", a, values.float()).reshape(batch, -1)[:, :d].to(dtype)
        logits = tk.linear(x + out.contiguous(), head)
        u = torch.rand(batch, generator=g).cuda()
        kw = dict(temperature=0.9, top_k=50, top_p=0.95, min_p=0.001)
        tokens, logprobs = tk.sample(logits, u, **kw)
        check(logits, u, tokens, logprobs, **kw)
        seen_tokens |= set(tokens.tolist())
    assert len(seen_tokens) > 10 and f32(0.9) != 0.9
    lengths = torch.full((batch,), slots, device="cuda")
    before = score.cpu().clone()
    ck, cv, cs, kept, left = tk.evict(keys, values, score, lengths, 6, recent=0)
    want, _ = evict64(dict(lengths=lengths.cpu()), 6, 0, before)
    assert torch.equal(kept.cpu(), want) and left.tolist() == [6] * batch
    assert torch.equal(ck.cpu(), keys.cpu().gather(2, want[..., None].expand(-1, -1, -1, dim)))
    assert torch.equal(positions.gather(2, kept).cpu(), positions.cpu().gather(2, want))
