"""What a language model does with a selection, measured: the next token out of its logits, tokens sorted by the experts
they were routed to and back, and the positions of a key-value cache that stay when it is full.

    sample              a token of each row, by temperature, min-p, top-k and top-p, from given random numbers
    dispatch            rows in the order of their experts
    combine             the way back, with weights (without them: dispatch's gradient)
    combine_backward    its gradients
    evict               the positions with the most accumulated attention weight and the recent ones, moved together
    replace_            the single-token form: a new token takes the slot with the least accumulated weight
"""
import math

import torch

own = False
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LOGITS = 256 * 131072            # the most logits of a drawn case
ROWS = 8192 * 8 * 2048           # the most values that a drawn case moves to or from experts
CACHE = 8 * 32768 * 32           # the most positions x queries of a drawn eviction


def listed():
    return [
        # One conversation: the next token of a single row, with the filters that an interactive session uses.
        dict(name="sample_one", op="sample", dtype="f32", rows=1, n=65536, temperature=0.8, top_k=64, top_p=0.95, min_p=0.0, per_row=False),
        # A serving batch: every request has parameters of its own; nucleus sampling without a limit on the count.
        dict(name="sample_batch", op="sample", dtype="bf16", rows=96, n=131072, temperature=1.0, top_k=0, top_p=0.9, min_p=0.0, per_row=True),
        # The largest batch, all filters at once.
        dict(name="sample_filters", op="sample", dtype="f32", rows=256, n=131072, temperature=0.9, top_k=200, top_p=0.95, min_p=0.01, per_row=False),
        # Plain draws from the whole distribution at a high temperature, over a vocabulary that divides by nothing.
        dict(name="sample_whole", op="sample", dtype="f32", rows=37, n=100003, temperature=1.5, top_k=0, top_p=1.0, min_p=0.0, per_row=False),
        # A decoding step's tokens sent to their experts: few rows, latency counts.
        dict(name="dispatch_step", op="dispatch", dtype="bf16", tokens=16, k=4, experts=64, d=4096, dropped=0.0),
        # A training batch's tokens sent to eight experts each.
        dict(name="dispatch_batch", op="dispatch", dtype="bf16", tokens=8192, k=8, experts=64, d=2048, dropped=0.0),
        # The same batch's results brought back with the router's weights.
        dict(name="combine_batch", op="combine", dtype="bf16", tokens=8192, k=8, experts=64, d=2048, dropped=0.0, weights=True),
        # The gradients of bringing back in f32, odd sizes, some tokens dropped for want of room.
        dict(name="combine_backward_ragged", op="combine_backward", dtype="f32", tokens=4093, k=6, experts=40, d=1001, dropped=0.05, weights=True),
        # A long prompt read: its cache cut down to what the last 32 queries and those before looked at.
        dict(name="evict_prompt", op="evict", dtype="bf16", batch=1, heads=8, group=4, queries=32, n=32768, dim=128, keep=4096, recent=512, ragged=False),
        # A batch of ragged conversations whose caches are cut together, in f32 with odd sizes; some are still short.
        dict(name="evict_ragged", op="evict", dtype="f32", batch=12, heads=4, group=2, queries=5, n=5001, dim=72, keep=1021, recent=63, ragged=True),
        # A decoding step of a batch whose caches are full: one slot of each head is given up.
        dict(name="replace_batch", op="replace", dtype="bf16", batch=64, heads=8, group=4, queries=1, n=4096, dim=128, recent=256, ragged=False),
        # A decoding step of one conversation.
        dict(name="replace_one", op="replace", dtype="f32", batch=1, heads=8, group=1, queries=1, n=2048, dim=64, recent=32, ragged=False),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "dispatch", "combine", "combine_backward", "evict", "replace"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "sample":
        rows, n = _spread(rng, 1, 256), _spread(rng, 1000, 131072)
        while rows * n > LOGITS:
            rows = max(1, rows // 2)
        return dict(op=op, dtype=dtype, rows=rows, n=n, temperature=rng.choice([0.0, 0.5, 0.7, 1.0, 1.0, 1.3, 2.0]),
                    top_k=rng.choice([0, 0, _spread(rng, 1, 1000), _spread(rng, 1, n)]), top_p=rng.choice([1.0, 0.5, 0.9, 0.97]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.2]), per_row=rng.random() < 0.5)
    if op in ("dispatch", "combine", "combine_backward"):
        while True:
            tokens, k, experts, d = _spread(rng, 1, 16384), _spread(rng, 1, 12), _spread(rng, 2, 512), _spread(rng, 64, 8192)
            d = -(-d // 64) * 64 if rng.random() < 0.6 else d
            size = 1 if dtype == "bf16" else 2
            if op == "combine_backward":
                size *= 2
            if tokens * min(k, experts) * d * size <= ROWS:
                break
        return dict(op=op, dtype=dtype, tokens=tokens, k=min(k, experts), experts=experts, d=d, dropped=rng.choice([0.0, 0.0, 0.1]),
                    weights=op == "combine_backward" or rng.random() < 0.6)
    while True:
        batch, heads, group, n = _spread(rng, 1, 64), _spread(rng, 1, 16), rng.choice([1, 2, 4, 7, 8]), _spread(rng, 64, 32768)
        queries = _spread(rng, 1, 64) if op == "evict" else 1
        if batch * heads * n * max(group * queries // 4, 4) <= CACHE:
            break
    case = dict(op=op, dtype=dtype, batch=batch, heads=heads, group=group, queries=queries, n=n, dim=rng.choice([64, 72, 80, 128, 256]))
    if op == "evict":
        case["keep"] = _spread(rng, 16, n)
        while batch * heads * case["keep"] * case["dim"] > ROWS // 8:
            case["keep"] //= 2
        case["recent"] = rng.randint(0, case["keep"] // 2)
    else:
        case["recent"] = rng.randint(0, n // 4)
    return dict(case, ragged=rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = dict(case=case)
    if case["op"] == "sample":
        rows, n = case["rows"], case["n"]
        # A broad bulk and a few tokens above it, by row from a confident prediction to an open one.
        x = torch.randn(rows, n, device="cuda", generator=g) * 2.0
        likely = torch.randint(0, n, (rows, 24), device="cuda", generator=g)
        s["logits"] = x.scatter_add_(1, likely, 14 * uniform(rows, 24) * uniform(rows, 1)).to(dt)
        s["u"] = uniform(rows)
        for name in ("temperature", "top_k", "top_p", "min_p"):
            s[name] = case[name]
        if case["per_row"]:
            s["temperature"] = case["temperature"] * (0.5 + uniform(rows))
            s["top_p"] = torch.where(uniform(rows) < 0.8, (case["top_p"] + 0.2 * (uniform(rows) - 0.5)).clamp(0.05, 1.0), 1.0)
            s["min_p"] = case["min_p"] * uniform(rows)
            most = max(case["top_k"], 1)
            s["top_k"] = (torch.randint(0, most, (rows,), device="cuda", generator=g) + (case["top_k"] > 0)).to(torch.int32)
        return s
    if "experts" in case:
        tokens, k, experts, d = case["tokens"], case["k"], case["experts"], case["d"]
        # Some experts are liked more than others.
        score = torch.randn(tokens, experts, device="cuda", generator=g) + 0.8 * torch.randn(experts, device="cuda", generator=g)
        top = score.topk(k, dim=1)
        s["idx"] = torch.where(uniform(tokens, k) < case["dropped"], -1, top.indices).contiguous()
        if case["op"] == "dispatch":
            s["x"] = normal(tokens, d)
            return s
        s["place"] = _sorted(s["idx"], experts)[0]
        s["weights"] = torch.softmax(top.values, 1).to(dt) if case["weights"] else None
        s["ys"] = normal(tokens * k, d)
        if case["op"] == "combine_backward":
            s["dy"] = normal(tokens, d)
        return s
    batch, heads, n, dim = case["batch"], case["heads"], case["n"], case["dim"]
    s["keys"], s["values"] = normal(batch, heads, n, dim), normal(batch, heads, n, dim)
    # Accumulated weight: most positions have little, a few a lot.
    s["score"] = (torch.randn(batch, heads, n, device="cuda", generator=g) * 1.5 - 3).exp()
    least = n // 3 if case["ragged"] else n
    s["lengths"] = torch.randint(least, n + 1, (batch,), device="cuda", generator=g)
    a = torch.randn(batch, heads * case["group"], case["queries"], n, device="cuda", generator=g) * 2.0
    a.masked_fill_(torch.arange(n, device="cuda") >= s["lengths"][:, None, None, None], -math.inf)
    s["weights"] = torch.softmax(a, -1).to(dt)
    if case["op"] == "replace":
        s["key"], s["value"] = normal(batch, heads, dim), normal(batch, heads, dim)
        # Slots hold the positions of a longer conversation in no order (a full cache), or the first ones in order.
        at = torch.rand(batch, heads, n, device="cuda", generator=g).argsort(-1)
        full = (s["lengths"] == n)[:, None, None]
        s["positions"] = torch.where(full, at + n, torch.arange(n, device="cuda"))
        s["lengths"] = torch.where(s["lengths"] == n, 2 * n, s["lengths"])
    return s


def _sorted(idx, experts):
    """(place, offsets, the flat places in their experts' order) of tokens x k experts; places out of range have none."""
    flat = idx.reshape(-1)
    held = (flat >= 0) & (flat < experts)
    order = torch.where(held, flat, experts).sort(stable=True).indices
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=idx.device)
    place = torch.where(held, place, -1).reshape(idx.shape)
    count = (flat[None] == torch.arange(experts, device=idx.device)[:, None]).sum(1)
    return place, torch.cat([count.new_zeros(1), count.cumsum(0)]), order


def _plain_sample(s):
    x, rows = s["logits"].float(), s["logits"].shape[0]

    def each(name):
        v = s[name]
        if not isinstance(v, torch.Tensor):
            v = torch.full((rows,), v, dtype=torch.int32 if name == "top_k" else torch.float32, device=x.device)
        return v[:, None] if name == "top_k" else v.double()[:, None]

    # (64 bits: a token is chosen by where a sum over the vocabulary passes a border)
    temperature, top_k, top_p, min_p = each("temperature"), each("top_k"), each("top_p"), each("min_p")
    x, order = x.sort(dim=1, descending=True, stable=True)
    x = x.double()
    d = x - x[:, :1]
    greedy = temperature <= 0
    w = torch.where(greedy, (d == 0).double(), torch.exp(d / torch.where(greedy, 1.0, temperature)))
    rank = torch.arange(x.shape[1], device=x.device)
    w = torch.where((w >= min_p) & ((top_k <= 0) | (rank < top_k)) & (~greedy | (rank < 1)), w, 0.0)
    before = w.cumsum(1) - w
    w = torch.where((before < top_p * w.sum(1, keepdim=True)) | (rank < 1), w, 0.0)
    total = w.sum(1, keepdim=True)
    at = ((w.cumsum(1) <= s["u"].double()[:, None] * total).sum(1, keepdim=True)).clamp(max=x.shape[1] - 1)
    at = torch.minimum(at, (w > 0).sum(1, keepdim=True) - 1)
    return {"tokens": order.gather(1, at)[:, 0], "logprobs": (w.gather(1, at) / total).log()[:, 0].float()}


def _plain_experts(s):
    case = s["case"]
    if case["op"] == "dispatch":
        place, offsets, order = _sorted(s["idx"], case["experts"])
        held = torch.arange(order.numel(), device=order.device) < offsets[-1]
        xs = torch.where(held[:, None], s["x"][order // case["k"]], torch.zeros((), dtype=s["x"].dtype, device=order.device))
        return {"xs": xs, "place": place, "offsets": offsets}
    place, dt = s["place"], s["ys"].dtype
    held = (place >= 0)[..., None]
    rows = torch.where(held, s["ys"].float()[place.clamp(min=0)], 0.0)
    w = None if s["weights"] is None else s["weights"].float()[..., None]
    if case["op"] == "combine":
        return (rows if w is None else rows * w).sum(1).to(dt)
    dy = s["dy"].float()
    dys = torch.zeros(s["ys"].shape, device=dy.device)
    t, j = (place >= 0).nonzero(as_tuple=True)
    dys[place[t, j]] = w[t, j] * dy[t]
    return {"dys": dys.to(dt), "dweights": (rows * dy[:, None]).sum(-1).to(dt)}


def _accumulated(s, lengths):
    """The score with the weights of a head's queries added, summed in 64 bits and rounded once."""
    batch, heads, n = s["score"].shape
    add = s["weights"].reshape(batch, heads, -1, n).sum(2, dtype=torch.float64)
    valid = torch.arange(n, device=add.device) < lengths[:, None, None]
    return torch.where(valid, s["score"].double() + add, s["score"].double()).float()


def _plain_evict(s):
    keep, recent, lengths = s["case"]["keep"], s["case"]["recent"], s["lengths"]
    score = _accumulated(s, lengths)
    n = score.shape[2]
    at = torch.arange(n, device=score.device)
    key = torch.where(at >= (lengths - recent)[:, None, None], math.inf, score)
    key = torch.where(at >= lengths[:, None, None], -math.inf, key)
    kept = key.sort(dim=2, descending=True, stable=True).indices[..., :keep]
    held = torch.arange(kept.shape[2], device=kept.device) < lengths[:, None, None]
    kept = torch.where(held, kept, n).sort(dim=2).values
    from_ = torch.where(held, kept, 0)

    def rows(t):
        got = t.gather(2, from_[..., None].expand(-1, -1, -1, t.shape[3]))
        return torch.where(held[..., None], got, torch.zeros((), dtype=t.dtype, device=t.device))

    return {"keys": rows(s["keys"]), "values": rows(s["values"]), "score": torch.where(held, score.gather(2, from_), 0.0),
            "kept": torch.where(held, kept, -1), "lengths": lengths.clamp(max=keep)}


def _plain_replace(s):
    seen, recent = s["lengths"][:, None, None], s["case"]["recent"]
    n = s["score"].shape[2]
    s["score"].copy_(_accumulated(s, s["lengths"]))
    key = torch.where(s["positions"] >= seen - recent, math.inf, s["score"])
    least = (key == key.min(dim=2, keepdim=True).values).int().argmax(2, keepdim=True)
    slot = torch.where(seen < n, seen, least)
    s["keys"].scatter_(2, slot[..., None].expand(-1, -1, -1, s["keys"].shape[3]), s["key"][:, :, None])
    s["values"].scatter_(2, slot[..., None].expand(-1, -1, -1, s["values"].shape[3]), s["value"][:, :, None])
    s["score"].scatter_(2, slot, 0.0)
    s["positions"].scatter_(2, slot, seen.expand_as(slot))
    return {"slots": slot[..., 0], **{k: s[k] for k in ("keys", "values", "score", "positions")}}


def _plain(s):
    op = s["case"]["op"]
    if op == "sample":
        return _plain_sample(s)
    if op == "evict":
        return _plain_evict(s)
    if op == "replace":
        return _plain_replace(s)
    return _plain_experts(s)


def _own(s):
    import top_selection_prof_gb300 as tk
    case = s["case"]
    op = case["op"]
    if op == "sample":
        tokens, logprobs = tk.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return {"tokens": tokens, "logprobs": logprobs}
    if op == "dispatch":
        xs, place, offsets = tk.dispatch(s["x"], s["idx"], case["experts"])
        return {"xs": xs, "place": place, "offsets": offsets}
    if op == "combine":
        return tk.combine(s["ys"], s["place"], s["weights"])
    if op == "combine_backward":
        dys, dweights = tk.combine_backward(s["dy"], s["ys"], s["place"], s["weights"])
        return {"dys": dys, "dweights": dweights}
    if op == "evict":
        keys, values, score, kept, lengths = tk.evict(s["keys"], s["values"], s["score"], s["lengths"], case["keep"], recent=case["recent"], weights=s["weights"])
        return {"keys": keys, "values": values, "score": score, "kept": kept, "lengths": lengths}
    slots = tk.replace_(s["keys"], s["values"], s["score"], s["positions"], s["lengths"], s["key"], s["value"], recent=case["recent"], weights=s["weights"])
    return {"slots": slots, **{k: s[k] for k in ("keys", "values", "score", "positions")}}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "sample":
        rows, n = case["rows"], case["n"]
        return {"bytes": rows * (size * n + 16 + (16 if case["per_row"] else 0)), "flops": 4 * rows * n}
    if "experts" in case:
        t, k, d = case["tokens"], case["k"], case["d"]
        if op == "dispatch":
            return {"bytes": size * d * (t + t * k) + 16 * t * k + 8 * (case["experts"] + 1), "flops": t * k}
        weights = size * t * k if case["weights"] else 0
        if op == "combine":
            return {"bytes": size * d * (t + t * k) + 8 * t * k + weights, "flops": 2 * t * k * d}
        return {"bytes": size * d * (t + 2 * t * k) + 8 * t * k + 2 * weights, "flops": 3 * t * k * d}
    rows, n, dim = case["batch"] * case["heads"], case["n"], case["dim"]
    read = n * 2 // 3 if case["ragged"] else n
    weights = size * rows * case["group"] * case["queries"] * read
    flops = rows * case["group"] * case["queries"] * read
    if op == "evict":
        kept = min(case["keep"], read)
        return {"bytes": weights + rows * (4 * read + kept * (4 * dim * size + 12)) + 16 * case["batch"], "flops": flops + rows * read}
    return {"bytes": weights + rows * (read * (8 + (8 if case["recent"] else 0)) + 4 * dim * size + 20) + 8 * case["batch"], "flops": flops + rows * read}


def _exact_sample(s):
    rows = s["logits"].shape[0]
    tokens, logprobs = [], []
    for r in range(rows):
        x = s["logits"][r].double()

        def of(name, kind):
            v = s[name]
            return kind(v[r]) if isinstance(v, torch.Tensor) else kind(torch.tensor(v, dtype=torch.float32 if kind is float else torch.int32))

        temperature, top_k = of("temperature", float), of("top_k", int)
        top_p, min_p, u = of("top_p", float), of("min_p", float), float(s["u"][r])
        best = int((x == x.max()).nonzero()[0])
        if temperature <= 0:
            tokens.append(best)
            logprobs.append(0.0)
            continue
        p = torch.softmax(x / temperature, 0)
        cand = (p >= min_p * p[best]).nonzero()[:, 0]
        cand = cand[torch.argsort(x[cand], descending=True, stable=True)]
        if top_k > 0:
            cand = cand[:top_k]
        cum = p[cand].cumsum(0)
        last = int(torch.searchsorted(cum, top_p * cum[-1])) if top_p < 1 else cand.numel() - 1
        cum = cum[:min(last, cand.numel() - 1) + 1]
        at = min(int(torch.searchsorted(cum, u * cum[-1], right=True)), cum.numel() - 1)
        tokens.append(int(cand[at]))
        logprobs.append(math.log(float(p[cand[at]] / cum[-1])))
    return {"tokens": torch.tensor(tokens, device="cuda"), "logprobs": torch.tensor(logprobs, dtype=torch.float64, device="cuda")}


def exact(case, seed):
    """The same in 64 bits, from the definitions: a row at a time, experts one after another, positions chosen on the host."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(s)
    if op == "dispatch":
        flat, k = s["idx"].reshape(-1), case["k"]
        runs = [(flat == e).nonzero()[:, 0] for e in range(case["experts"])]
        order = torch.cat(runs)
        xs = torch.zeros(flat.numel(), case["d"], dtype=torch.float64, device="cuda")
        xs[:order.numel()] = s["x"].double()[torch.div(order, k, rounding_mode="floor")]
        place = torch.full_like(flat, -1)
        place[order] = torch.arange(order.numel(), device="cuda")
        offsets = torch.tensor([0] + [r.numel() for r in runs], device="cuda").cumsum(0)
        return {"xs": xs, "place": place.reshape(s["idx"].shape), "offsets": offsets}
    if op in ("combine", "combine_backward"):
        place, ys = s["place"], s["ys"].double()
        w = torch.ones(place.shape, dtype=torch.float64, device="cuda") if s["weights"] is None else s["weights"].double()
        y = torch.zeros(place.shape[0], ys.shape[1], dtype=torch.float64, device="cuda")
        dys, dw = torch.zeros_like(ys), torch.zeros_like(w)
        for j in range(place.shape[1]):
            t = (place[:, j] >= 0).nonzero()[:, 0]
            r = place[t, j]
            if op == "combine":
                y[t] += w[t, j][:, None] * ys[r]
            else:
                dy = s["dy"].double()[t]
                dys[r] += w[t, j][:, None] * dy
                dw[t, j] = torch.linalg.vecdot(dy, ys[r])
        return y if op == "combine" else {"dys": dys, "dweights": dw}
    lengths = s["lengths"].tolist()
    batch, heads, n = s["score"].shape
    group, score = case["group"], s["score"].double()
    for b in range(batch):
        m = min(lengths[b], n)
        for h in range(heads):
            score[b, h, :m] += s["weights"][b, h * group:(h + 1) * group, :, :m].double().sum((0, 1))
    score = score.float()       # (what is accumulated is held in 32 bits, and chosen by as it is held)
    if op == "replace":
        slots = torch.empty(batch, heads, dtype=torch.int64, device="cuda")
        for b in range(batch):
            for h in range(heads):
                slot = lengths[b]
                if slot >= n:
                    may = (s["positions"][b, h] < lengths[b] - case["recent"]).nonzero()[:, 0]
                    slot = int(may[torch.argsort(score[b, h, may], stable=True)[0]])
                slots[b, h] = slot
                s["keys"][b, h, slot], s["values"][b, h, slot] = s["key"][b, h], s["value"][b, h]
                score[b, h, slot], s["positions"][b, h, slot] = 0.0, lengths[b]
        return {"slots": slots, "keys": s["keys"].double(), "values": s["values"].double(), "score": score.double(), "positions": s["positions"]}
    keep, recent = case["keep"], case["recent"]
    out = {k: torch.zeros(batch, heads, keep, case["dim"], dtype=torch.float64, device="cuda") for k in ("keys", "values")}
    out["score"] = torch.zeros(batch, heads, keep, dtype=torch.float64, device="cuda")
    out["kept"] = torch.full((batch, heads, keep), -1, device="cuda")
    for b in range(batch):
        m = lengths[b]
        old = max(m - recent, 0)
        for h in range(heads):
            at = torch.arange(m, device="cuda")
            if m > keep:
                best = torch.argsort(score[b, h, :old], descending=True, stable=True)[:keep - (m - old)]
                at = torch.cat([best.sort().values, at[old:]])
            out["keys"][b, h, :at.numel()], out["values"][b, h, :at.numel()] = s["keys"][b, h, at].double(), s["values"][b, h, at].double()
            out["score"][b, h, :at.numel()], out["kept"][b, h, :at.numel()] = score[b, h, at].double(), at
    return {**out, "lengths": torch.tensor([min(m, keep) for m in lengths], device="cuda")}
