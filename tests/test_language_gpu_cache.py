"""What stays in a cache, and one token put into a full one, on the GPU against plain forms on the CPU in 64 bits.

Weights that are multiples of 2^-8 with small sums give scores that f32 holds exactly, with many equal ones: choices and
moved rows are compared bit for bit.  Other weights are summed to about 2^-44 of the sum of their magnitudes and rounded
once: a score is off by half a step (2^-24 of it) and that.
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


def case(batch, heads, group, queries, n, kd, vd, dtype, seed, wdtype=None, exact=True):
    g = gen(seed)
    s = dict(keys=torch.randn(batch, heads, n, kd, generator=g).to(dtype), values=torch.randn(batch, heads, n, vd, generator=g).to(dtype))
    lengths = torch.randint(0, n + 1, (batch,), generator=g)
    lengths[0] = n
    if batch > 2:
        lengths[1], lengths[2] = 0, 1
    s["lengths"] = lengths
    if exact:
        s["score"] = torch.randint(0, 200, (batch, heads, n), generator=g).float() / 16
        w = torch.randint(0, 30, (batch, heads * group, queries, n), generator=g) / 256
    else:
        s["score"] = torch.rand(batch, heads, n, generator=g) ** 6
        w = torch.softmax(3 * torch.randn(batch, heads * group, queries, n, generator=g), -1)
    s["weights"] = w.to(wdtype or dtype) if queries else None
    return s


def added(s):
    """score + weights, in 64 bits, where there is a token; NaN weights are 0."""
    score = s["score"].double()
    if s["weights"] is None:
        return score
    b, h, n = score.shape
    w = s["weights"].double().nan_to_num(nan=0.0, posinf=torch.inf, neginf=-torch.inf).reshape(b, h, -1, n).sum(2)
    held = torch.arange(n) < s["lengths"].clamp(0, n)[:, None, None]
    return torch.where(held, score + w, score)


def evict64(s, keep, recent, score):
    """(kept, lengths) from scores in f32."""
    b, h, n = score.shape
    kept = torch.full((b, h, keep), -1)
    lengths = s["lengths"].clamp(0, n)
    for i in range(b):
        m = int(lengths[i])
        old = max(m - recent, 0)
        for j in range(h):
            if m <= keep:
                at = torch.arange(m)
            else:
                x = score[i, j, :old].double()
                x = torch.where(x.isnan(), torch.inf, torch.where(x == torch.inf, 1e300, x))   # (NaN above infinity)
                at = torch.cat([x.sort(descending=True, stable=True).indices[:keep - (m - old)].sort().values, torch.arange(old, m)])
            kept[i, j, :at.numel()] = at
    return kept, lengths.clamp(max=keep)


def cuda(s):
    return {k: v if v is None else v.cuda() for k, v in s.items()}


def check_evict(tk, s, keep, recent, on=None, exact=True):
    on = on or cuda(s)
    got = tk.evict(on["keys"], on["values"], on["score"], on["lengths"], keep, recent=recent, weights=on["weights"])
    keys, values, score, kept, lengths = (t.cpu() for t in got)
    full = added(s)
    want, want_lengths = evict64(s, keep, recent, full.float())
    assert torch.equal(lengths, want_lengths)
    if exact:
        assert torch.equal(kept, want)
    else:
        # another choice only among scores that a rounding away from the last one kept
        for i, j in (kept != want).any(-1).nonzero().tolist():
            a, b = set(kept[i, j].tolist()), set(want[i, j].tolist())
            last = full[i, j, list(b)].min()
            assert all(abs(float(full[i, j, p] - last)) <= 2.0 ** -22 * float(last) for p in a ^ b)
    held = (kept >= 0)
    at = kept.clamp(min=0)
    for out, src in ((keys, s["keys"]), (values, s["values"])):
        rows = src.gather(2, at[..., None].expand(-1, -1, -1, src.shape[3]))
        assert torch.equal(out, torch.where(held[..., None], rows, torch.zeros((), dtype=rows.dtype)))
    ref = torch.where(held, full.gather(2, at), 0.0)
    if exact:
        assert torch.equal(score.nan_to_num(7.0), ref.float().nan_to_num(7.0))
    else:
        assert bool(((score.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 2.0 ** -40 * (ref.abs() + 1e-30)).all())
    return got


SIZES = [(1, 1, 1, 1, 1, 8, 8, 1, 0), (3, 2, 1, 1, 40, 64, 64, 16, 4), (4, 2, 4, 3, 333, 72, 40, 100, 100), (2, 3, 2, 33, 2050, 33, 7, 777, 0),
         (5, 1, 7, 5, 6000, 80, 80, 1024, 1), (1, 2, 2, 2, 20_001, 16, 16, 5000, 300), (3, 8, 1, 0, 513, 128, 64, 600, 5),
         (40, 8, 1, 1, 700, 8, 8, 64, 32), (1, 1, 1, 1, 100_000, 8, 8, 1, 0), (1, 1, 1, 2, 70_000, 8, 16, 60_000, 59_000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,heads,group,queries,n,kd,vd,keep,recent", SIZES)
def test_evict(tk, batch, heads, group, queries, n, kd, vd, keep, recent, dtype):
    check_evict(tk, case(batch, heads, group, queries, n, kd, vd, dtype, n), keep, recent)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [7, 31, 32, 33, 63, 64, 65, 80, 127, 128, 129, 136])
@pytest.mark.parametrize("group,queries", [(8, 60), (1, 33), (3, 1)])
def test_evict_of_few_positions(tk, n, group, queries, dtype):
    check_evict(tk, case(3, 2, group, queries, n, 16, 8, dtype, n + queries), max(1, n // 2), n // 8)


@pytest.mark.parametrize("wdtype", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1000, 9001])
def test_evict_by_attention(tk, n, dtype, wdtype):
    check_evict(tk, case(4, 2, 4, 17, n, 32, 32, dtype, n, wdtype, exact=False), n // 3, 50, exact=False)


def test_sums_are_exact_to_their_rounding(tk):
    """One large and many small weights, in an order that f32 sums would lose the small ones in."""
    n, queries = 300, 200
    s = case(1, 1, 4, queries, n, 8, 8, torch.float32, 1)
    w = torch.full((1, 4, queries, n), 2.0 ** -25)
    w[0, 0, 0] = 1.0
    s["weights"], s["score"] = w, torch.zeros(1, 1, n)
    got = check_evict(tk, s, n, 0)
    assert float(got[2][0, 0, 5]) == float(torch.tensor(1.0 + 799 * 2.0 ** -25, dtype=torch.float64).float())


@pytest.mark.parametrize("op,rows", [("evict", 1 << 18), ("evict", 4096), ("replace", 1 << 16), ("replace", 1 << 14)])
@pytest.mark.parametrize("n", [63, 70, 72])
def test_sums_of_many_rows(tk, op, rows, n):
    """Ones (a row of each thread's, or the score) and rows of 2^-26 with some bits behind, which the sums' second parts would round
    away as they grow.  A sum of K rows at a time rounds off at most (K + 3) / 2 of 2^-48 of the magnitudes' sum a row, 5.5 with
    K = 8, and joining 32 parts 8 of them each: (rows + 32) 2^-45 in all, and half a step."""
    w = (2.0 ** -26 + 2.0 ** -37 * (0.5 + torch.arange(n, dtype=torch.float64) / (2 * n))).float()
    s = case(1, 1, 8, 0, n, 8, 8, torch.float32, 1)
    s["score"], s["lengths"] = torch.ones(1, 1, n), torch.tensor([n])
    on = cuda(s)
    on["weights"] = w.cuda().expand(1, 8, rows // 8, n).contiguous()
    ones = 8 if op == "evict" else 0
    on["weights"].view(rows, n)[:ones] = 1.0
    want = 1.0 + ones + (rows - ones) * w.double()
    if op == "evict":
        got = tk.evict(on["keys"], on["values"], on["score"], on["lengths"], n, weights=on["weights"])[2][0, 0].cpu()
    else:
        positions, key, value = torch.arange(n).expand(1, 1, n).contiguous().cuda(), on["keys"][:, :, 0].clone(), on["values"][:, :, 0].clone()
        slot = tk.replace_(on["keys"], on["values"], on["score"], positions, on["lengths"], key, value, weights=on["weights"])
        got = on["score"][0, 0].cpu()
        assert float(got[int(slot)]) == 0.0
        want[int(slot)] = 0.0
    bound = 2.0 ** -24 * want + (rows + 32) * 2.0 ** -45 * want
    assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound.clamp(min=1e-30)).max())


def test_scores_and_weights_that_are_not_numbers(tk):
    for dtype in DTYPES:
        s = case(2, 1, 2, 3, 500, 16, 16, dtype, 2)
        s["lengths"][1] = 400
        s["weights"][0, 1, 2] = torch.nan          # a query whose mask left nothing
        s["weights"][1, :, :, 400:] = torch.nan    # behind the length
        s["weights"][1, 0, 1, 405] = torch.inf
        s["weights"][1, 0, 1, 3] = torch.inf
        s["score"][0, 0, 7], s["score"][0, 0, 9], s["score"][1, 0, 450] = torch.nan, -torch.inf, torch.inf
        for keep, recent in ((100, 10), (2, 1), (499, 0), (500, 500)):
            check_evict(tk, s, keep, recent)


def test_lengths_out_of_range_and_few_kept(tk):
    s = case(4, 2, 1, 2, 100, 16, 16, torch.float32, 3)
    s["lengths"] = torch.tensor([-5, 1 << 40, 100, 37])
    for keep, recent in ((1, 0), (1, 1), (36, 36), (37, 3), (38, 0), (200, 150)):
        check_evict(tk, s, keep, recent)
    s["score"][:] = 0.25
    s["weights"] = None
    check_evict(tk, s, 20, 5)      # all equal: the first ones stay


@pytest.mark.parametrize("dtype", DTYPES)
def test_caches_laid_out_otherwise(tk, dtype):
    """Positions before heads, keys and values in one buffer, rows and weights that start off 16-byte boundaries."""
    s = case(3, 4, 2, 3, 301, 64, 64, dtype, 4)
    on = cuda(s)
    on["keys"] = on["keys"].transpose(1, 2).contiguous().transpose(1, 2)
    both = torch.zeros(3, 4, 301, 131, dtype=dtype, device="cuda")
    on["values"] = both[..., 65:129].copy_(on["values"])
    on["score"] = torch.zeros(3, 5, 304, device="cuda")[:, 1:, 3:].copy_(on["score"])
    on["weights"] = torch.zeros(3, 8, 4, 303, dtype=dtype, device="cuda")[:, :, 1:, 1:302].copy_(on["weights"])
    check_evict(tk, s, 100, 20, on)
    s["weights"] = s["weights"][:, :1, :1].expand(-1, 8, 3, -1)
    on["weights"] = s["weights"][:, :1, :1].cuda().expand(-1, 8, 3, -1)
    check_evict(tk, s, 100, 20, on)


# ---- one token --------------------------------------------------------------------
def replace64(s, recent):
    """The state after the call, and the slots."""
    n = s["score"].shape[2]
    score = added(s).float()
    out = {k: v.clone() for k, v in s.items() if k in ("keys", "values", "positions")}
    slots = torch.empty(score.shape[:2], dtype=torch.int64)
    for b in range(score.shape[0]):
        seen = max(int(s["lengths"][b]), 0)
        for h in range(score.shape[1]):
            slot = seen
            if seen >= n:
                may = (s["positions"][b, h] < seen - recent).nonzero()[:, 0] if recent else torch.arange(n)
                x = score[b, h, may].double()
                x = torch.where(x.isnan(), torch.inf, torch.where(x == torch.inf, 1e300, x))
                slot = int(may[x.sort(stable=True).indices[0]]) if may.numel() else -1
            slots[b, h] = slot
            if slot >= 0:
                out["keys"][b, h, slot], out["values"][b, h, slot] = s["key"][b, h], s["value"][b, h]
                score[b, h, slot], out["positions"][b, h, slot] = 0.0, seen
    return {**out, "score": score}, slots


def step(batch, heads, group, n, kd, vd, dtype, seed, queries=1, wdtype=None):
    s = case(batch, heads, group, queries, n, kd, vd, dtype, seed, wdtype)
    g = gen(seed + 1)
    s["lengths"][::2] = 2 * n + torch.randint(0, 5, s["lengths"][::2].shape, generator=g)
    s["positions"] = torch.argsort(torch.rand(batch, heads, n, generator=g), -1) + n
    s["key"], s["value"] = torch.randn(batch, heads, kd, generator=g).to(dtype), torch.randn(batch, heads, vd, generator=g).to(dtype)
    return s


def check_replace(tk, s, recent, on=None):
    on = on or cuda(s)
    want, slots = replace64(s, recent)
    got = tk.replace_(on["keys"], on["values"], on["score"], on["positions"], on["lengths"], on["key"], on["value"], recent=recent,
                      weights=on["weights"])
    assert torch.equal(got.cpu(), slots)
    for k, v in want.items():
        assert torch.equal(on[k].cpu().nan_to_num(7.0) if v.is_floating_point() else on[k].cpu(), v.nan_to_num(7.0) if v.is_floating_point() else v), k


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,heads,group,n,kd,vd,recent", [(1, 1, 1, 1, 8, 8, 0), (4, 3, 2, 50, 72, 40, 10), (5, 8, 4, 1024, 128, 128, 64),
                                                              (1, 8, 1, 4097, 64, 33, 0), (70, 8, 2, 300, 16, 16, 299), (2, 1, 8, 40_001, 8, 8, 100)])
def test_replace(tk, batch, heads, group, n, kd, vd, recent, dtype):
    for queries in (1, 0, 3):
        check_replace(tk, step(batch, heads, group, n, kd, vd, dtype, n + queries, queries), recent)
    check_replace(tk, step(batch, heads, group, n, kd, vd, dtype, n, 1, DTYPES[dtype == DTYPES[0]]), recent)


def test_replace_where_nothing_may_go_and_not_numbers(tk):
    s = step(3, 2, 1, 60, 16, 16, torch.float32, 5)
    s["lengths"] = torch.tensor([200, 60, 59])
    s["positions"][0, 0] = torch.arange(140, 200)            # all recent
    s["positions"][1] = torch.arange(60)                     # as many tokens as slots
    s["score"][0, 1, :] = torch.nan
    s["score"][0, 1, 33], s["score"][0, 1, 12] = torch.inf, torch.inf
    s["score"][1, 0, 5] = -torch.inf
    s["weights"][1, 0, 0] = torch.nan
    check_replace(tk, s, 59)
    check_replace(tk, s, 20)
    check_replace(tk, s, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [61, 64, 4096, 4097])
@pytest.mark.parametrize("recent", [0, 1, 7])
def test_positions_behind_the_length_stay(tk, n, recent, dtype):
    """A slot whose position is not below lengths - recent is never given up, with recent 0 neither: tokens that were taken back, or
    slots that are held by a large position."""
    s = step(4, 2, 2, n, 16, 16, dtype, n)
    g = gen(n)
    s["positions"] = torch.argsort(torch.rand(4, 2, 2 * n, generator=g), -1)[..., :n].contiguous()
    s["lengths"] = torch.tensor([n, n + 5, 2 * n, n])
    s["positions"][3, 0] += n                                # none of its slots may go
    s["positions"][3, 1] += n
    s["positions"][3, 1, n // 2] = n - 1 - recent            # one
    on = cuda(s)
    score, want = added(s).float(), torch.empty(4, 2, dtype=torch.int64)
    for b in range(4):
        for h in range(2):
            may = (s["positions"][b, h] < int(s["lengths"][b]) - recent).nonzero()[:, 0]
            want[b, h] = may[score[b, h, may].sort(stable=True).indices[0]] if may.numel() else -1
    assert want[3].tolist() == [-1, n // 2]
    got = tk.replace_(*(on[k] for k in ("keys", "values", "score", "positions", "lengths", "key", "value")), recent=recent, weights=on["weights"])
    assert torch.equal(got.cpu(), want)
    for b in range(4):
        for h in range(2):
            slot = int(want[b, h])
            if slot >= 0:
                s["keys"][b, h, slot], s["values"][b, h, slot] = s["key"][b, h], s["value"][b, h]
                score[b, h, slot], s["positions"][b, h, slot] = 0.0, s["lengths"][b]
    assert torch.equal(on["score"].cpu(), score) and all(torch.equal(on[k].cpu(), s[k]) for k in ("keys", "values", "positions"))


def test_replace_in_one_buffer(tk):
    s = step(3, 4, 2, 64, 32, 32, torch.bfloat16, 6)
    on = cuda(s)
    both = torch.cat([on["keys"], on["values"]], -1).transpose(1, 2).contiguous().transpose(1, 2)
    on["keys"], on["values"] = both[..., :32], both[..., 32:]
    check_replace(tk, s, 8, on)


@pytest.mark.parametrize("dim", [0, 1, 2, 3, 4])
def test_keys_and_values_stacked(tk, dim):
    s = step(3, 4, 2, 64, 32, 32, torch.bfloat16, 9)
    on = cuda(s)
    on["keys"], on["values"] = torch.stack([on["keys"], on["values"]], dim).unbind(dim) if dim < 4 else (
        torch.cat([on["keys"], on["values"]], -1).split(32, -1))
    check_replace(tk, s, 8, on)
    state, _ = replace64(s, 8)
    s.update(state)
    s["lengths"], s["weights"] = torch.tensor([64, 30, 64]), None
    on["lengths"], on["weights"] = s["lengths"].cuda(), None
    check_evict(tk, s, 20, 4, on)


def test_a_conversation_past_its_cache(tk):
    """Token after token into a cache of 24 slots, then cut to 10: what is held is always what the definition holds."""
    g = gen(7)
    n, total = 24, 60
    s = dict(keys=torch.zeros(1, 2, n, 8), values=torch.zeros(1, 2, n, 8), score=torch.zeros(1, 2, n), positions=torch.zeros(1, 2, n, dtype=torch.int64))
    on = cuda(s)
    for t in range(total):
        new = dict(lengths=torch.tensor([t]), key=torch.full((1, 2, 8), float(t)), value=torch.full((1, 2, 8), -float(t)),
                   weights=torch.randint(0, 99, (1, 4, 1, n), generator=g) / 64)
        s.update(new), on.update(cuda(new))
        check_replace(tk, s, 5, on)
        state, _ = replace64(s, 5)
        s.update(state)
    assert torch.equal(s["keys"][0, :, :, 0].long(), s["positions"][0])
    assert all(set(range(total - 6, total)) <= set(row.tolist()) for row in s["positions"][0])
    s["lengths"], s["weights"] = torch.tensor([n]), None
    check_evict(tk, s, 10, 0)


def test_capture_and_streams(tk):
    a, b = (case(3, 2, 2, 5, 3000, 64, 64, torch.bfloat16, seed) for seed in (8, 9))
    A, B = cuda(a), cuda(b)

    def run(s, stream=None):
        return tk.evict(s["keys"], s["values"], s["score"], s["lengths"], 500, recent=20, weights=s["weights"], stream=stream)

    want = [run(A), run(B)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(A, side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(A)
    for k in A:
        A[k].copy_(B[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want[1]))
    s = step(2, 2, 1, 100, 16, 16, torch.float32, 10)
    on = cuda(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots = tk.replace_(*(on[k] for k in ("keys", "values", "score", "positions", "lengths", "key", "value")), recent=3, weights=on["weights"])
    graph.replay()
    torch.cuda.synchronize()
    state, at = replace64(s, 3)
    assert torch.equal(slots.cpu(), at) and all(torch.equal(on[k].cpu(), v) for k, v in state.items())
    assert tk.evict(B["keys"][:0], B["values"][:0], B["score"][:0], B["lengths"][:0], 5)[0].shape == (0, 2, 5, 64)


def test_a_backward_pass_that_saved_a_cache_raises(tk):
    """replace_ counts as an in-place change of its four tensors and of what they are views of, and of nothing else."""
    names = ("keys", "values", "score", "positions", "lengths", "key", "value")
    s = cuda(step(2, 2, 1, 64, 32, 32, torch.float32, 12))
    both = torch.cat([s["keys"], s["values"]], -1)
    s["keys"], s["values"] = both[..., :32], both[..., 32:]

    def call(recent=3):
        return tk.replace_(*(s[k] for k in names), recent=recent, weights=s["weights"])

    for k in ("keys", "values", "score", "positions"):
        x = torch.ones(s[k].shape, device="cuda", requires_grad=True)
        y = x.gather(-1, s[k].clamp_(0, 63)) if k == "positions" else x * s[k]     # (what the product, the gather saved)
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    x = torch.ones(s["key"].shape, device="cuda", requires_grad=True)
    (x * s["key"] * s["value"]).sum().backward(inputs=[x])
    before = {k: s[k]._version for k in names}
    y = x * s["key"]
    call()
    y.sum().backward()
    after = {k: s[k]._version for k in names}
    assert [after[k] - before[k] for k in names] == [2, 2, 1, 1, 0, 0, 0]   # (keys and values share one buffer's count)
    with pytest.raises(tk.TopkError):
        call(recent=64)
    assert {k: s[k]._version for k in names} == after
    with torch.inference_mode():
        s = {k: v.clone() for k, v in s.items()}
        want = call()
    assert call().shape == want.shape


def test_refusals(tk):
    s = cuda(step(2, 2, 1, 50, 8, 8, torch.float32, 11))

    def evict(keep=10, recent=0, **kw):
        a = {**s, **kw}
        return tk.evict(a["keys"], a["values"], a["score"], a["lengths"], keep, recent=recent, weights=a["weights"])

    def replace(recent=0, **kw):
        a = {**s, **kw}
        return tk.replace_(*(a[k] for k in ("keys", "values", "score", "positions", "lengths", "key", "value")), recent=recent, weights=a["weights"])

    for call in (lambda: evict(keep=0), lambda: evict(recent=11), lambda: evict(recent=-1), lambda: replace(recent=50), lambda: replace(recent=-1),
                 lambda: replace(keys=s["values"]), lambda: replace(keys=s["keys"][:, :1].expand(-1, 2, -1, -1)), lambda: replace(key=s["keys"][:, :, 3])):
        with pytest.raises(tk.TopkError) as e:
            call()
        assert e.value.status == -1
    for kind, kw in ((ValueError, dict(score=s["score"][:, :1])), (TypeError, dict(score=s["score"].double())), (TypeError, dict(lengths=s["lengths"].int())),
                     (TypeError, dict(values=s["values"].bfloat16())), (ValueError, dict(weights=s["weights"][..., :40])),
                     (ValueError, dict(weights=torch.zeros(2, 3, 1, 50, device="cuda"))), (TypeError, dict(weights=s["weights"].double())),
                     (ValueError, dict(keys=s["keys"][0])), (ValueError, dict(keys=s["keys"].transpose(2, 3)))):
        with pytest.raises(kind):
            evict(**kw)
        with pytest.raises(kind):
            replace(**kw)
