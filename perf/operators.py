"""The operators around the selection in a sparse autoencoder's training step: the cases they are measured on,
their plain forms in elementary torch operations, and the calls a user makes of the framework.

    linear                    y = act(x W^T + b) + residual              (the encoder)
    linear_backward           its gradients, for every output
    linear_backward_selected  its gradients where only selected outputs carry one (BatchTopK)
    decode                    y[r] = b + sum of v_s W[c_s] over the selected (r, c_s)
    decode_backward           its gradients
    clip_grad_norm            the global norm over many tensors, and clipping
"""
import math

import torch

own = False
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MACS = 4096 * 512 * 65536        # the encoder of the BatchTopK workload: the most products a drawn case has
CLIP = 2 * 65536 * 512           # parameters of the largest autoencoder here


def listed():
    return [
        # One token's activations through the encoder of a 12288-feature dictionary: an interactive probe of a model.
        dict(name="encode_token", op="linear", dtype="bf16", rows=1, inner=512, outer=12288, act="relu", residual=False),
        # The BatchTopK workload's own activations, 4096 x 65536, being made: a training step's encoder.
        dict(name="encode_batch", op="linear", dtype="bf16", rows=4096, inner=512, outer=65536, act="relu", residual=False),
        # A layer in f32 with sizes that divide by nothing, its residual added: a skip connection around a dictionary.
        dict(name="linear_ragged_f32", op="linear", dtype="f32", rows=1003, inner=769, outer=5001, act="gelu", residual=True),
        # The dense gradient of an encoder with 12288 features, a batch of a training step.
        dict(name="linear_backward_batch", op="linear_backward", dtype="bf16", rows=4096, inner=512, outer=12288, act="relu", residual=False),
        # A wide layer's gradient: activations of width 4096, a batch that is not a power of two.
        dict(name="linear_backward_wide", op="linear_backward", dtype="bf16", rows=2000, inner=4096, outer=16384, act="silu", residual=False),
        # The encoder's gradient in a BatchTopK step: 32 of 65536 features a token carry one.
        dict(name="selected_backward_batch", op="linear_backward_selected", dtype="bf16", rows=4096, inner=512, outer=65536, k=131072, per_row=False, skew=3.0),
        # One token's reconstruction from its 64 largest features (selected per row).
        dict(name="decode_token", op="decode", dtype="bf16", rows=1, inner=512, outer=12288, k=64, per_row=True, skew=1.0),
        # The reconstruction of a whole BatchTopK batch.
        dict(name="decode_batch", op="decode", dtype="bf16", rows=4096, inner=512, outer=65536, k=131072, per_row=False, skew=3.0),
        # Its gradient: dictionary, values and bias.
        dict(name="decode_backward_batch", op="decode_backward", dtype="bf16", rows=4096, inner=512, outer=65536, k=131072, per_row=False, skew=3.0),
        # The same in f32 with odd sizes, where few features fire on most tokens.
        dict(name="decode_backward_skewed_f32", op="decode_backward", dtype="f32", rows=1001, inner=771, outer=12289, k=40013, per_row=False, skew=8.0),
        # The gradients of a small head: a few tensors, odd sizes.
        dict(name="clip_small", op="clip_grad_norm", dtype="f32", tensors=7, total=20011, clips=True),
        # All gradients of the autoencoder with 65536 features.
        dict(name="clip_autoencoder", op="clip_grad_norm", dtype="bf16", tensors=4, total=CLIP, clips=True),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_backward", "linear_backward_selected", "decode", "decode_backward", "clip_grad_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip_grad_norm":
        return dict(op=op, dtype=dtype, tensors=_spread(rng, 1, 300), total=_spread(rng, 1000, CLIP if dtype == "bf16" else CLIP // 2), clips=rng.random() < 0.75)
    if op.startswith("linear") and op != "linear_backward_selected":
        most = MACS if op == "linear" else MACS // 2
        most = most if dtype == "bf16" else most // 16
        while True:
            rows, inner, outer = _spread(rng, 1, 4096), _spread(rng, 64, 4096), _spread(rng, 64, 65536)
            if rng.random() < 0.5:
                inner, outer = -(-inner // 320) * 320, -(-outer // 320) * 320
            if rows * inner * outer <= most:
                break
        return dict(op=op, dtype=dtype, rows=rows, inner=inner, outer=outer, act=rng.choice(["none", "relu", "gelu", "silu"]), residual=op == "linear" and rng.random() < 0.4)
    rows, inner, outer = _spread(rng, 1, 4096), _spread(rng, 64, 2048), _spread(rng, 1000, 65536)
    while inner * outer > 65536 * 512:
        inner = max(64, inner // 2)
    per_row = rng.random() < 0.4
    k = _spread(rng, 1, 128) if per_row else max(1, min(131072, int(rows * math.exp(rng.uniform(0.0, math.log(64))))))
    k = min(k, outer // 8)
    if op != "decode":
        per_row = False if rng.random() < 0.5 else per_row
    return dict(op=op, dtype=dtype, rows=rows, inner=inner, outer=outer, k=k, per_row=per_row, skew=rng.choice([1.0, 2.0, 3.0, 6.0]))


def _sizes(case):
    """Elements of each gradient: a few large tensors and many small ones, with the given total."""
    n, total = case["tensors"], case["total"]
    n = min(n, total)
    share = [1.0 / (i // 2 + 1) ** 4 + 1e-6 for i in range(n)]
    sizes = [max(1, int((total - n) * s / sum(share))) for s in share]
    sizes[0] += total - sum(sizes)
    return sizes


def _places(case, g):
    """Distinct selected places, the features drawn with a skew, in no order of place (a selection lists them by value)."""
    rows, outer, k, skew = case["rows"], case["outer"], case["k"], case["skew"]
    if case["per_row"]:
        key = torch.rand(rows, outer, device="cuda", generator=g) ** (1.0 / skew)
        return (key * (1.0 - 0.5 * torch.arange(outer, device="cuda") / outer)).topk(k, dim=1).indices
    r = torch.randint(0, rows, (8 * k,), device="cuda", generator=g)
    c = (outer * torch.rand(8 * k, device="cuda", generator=g, dtype=torch.float64) ** skew).long().clamp_(max=outer - 1)
    flat = torch.unique(r * outer + c)
    if flat.numel() < k:
        flat = torch.randperm(rows * outer, device="cuda", generator=g)
    return flat[torch.randperm(flat.numel(), device="cuda", generator=g)[:k]].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

    if case["op"] == "clip_grad_norm":
        sizes = _sizes(case)
        grads = [normal(n, scale=0.01) for n in sizes]
        norm = 0.01 * math.sqrt(sum(sizes))
        return dict(case=case, grads=grads, out=[torch.empty_like(t) for t in grads], max_norm=norm * (0.3 if case["clips"] else 3.0))
    rows, inner, outer = case["rows"], case["inner"], case["outer"]
    s = dict(case=case, w=normal(outer, inner, scale=inner ** -0.5))
    if case["op"] in ("linear", "linear_backward"):
        s["x"], s["bias"] = normal(rows, inner), normal(outer, scale=0.1)
        if case["op"] == "linear":
            s["residual"] = normal(rows, outer) if case["residual"] else None
        else:
            s["dy"] = normal(rows, outer)
            s["pre"] = None if case["act"] == "none" else (s["x"].float() @ s["w"].float().T + s["bias"].float()).to(dt)
        return s
    s["idx"] = _places(case, g)
    s["vals"] = normal(*s["idx"].shape).abs().sort(dim=-1, descending=True).values.contiguous()
    if case["op"] == "decode":
        s["bias"] = normal(inner)
    elif case["op"] == "decode_backward":
        s["dy"] = normal(rows, inner)
    else:
        s["x"], s["dvals"] = normal(rows, inner), normal(*s["idx"].shape)
    return s


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _rows_cols(case, idx):
    if case["per_row"]:
        r = torch.arange(case["rows"], device=idx.device)[:, None].expand_as(idx)
        return r.reshape(-1), idx.reshape(-1)
    return idx // case["outer"], idx % case["outer"]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "clip_grad_norm":
        norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
        scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1)
        return {"norm": norm, "grads": [(t.float() * scale).to(t.dtype) for t in s["grads"]]}
    dt, w = s["w"].dtype, s["w"].float()
    if op == "linear":
        y = _act(s["x"].float() @ w.T + s["bias"].float(), case["act"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(dt)
    if op == "linear_backward":
        dz = s["dy"].float()
        dz = dz if s["pre"] is None else dz * _slope(s["pre"].float(), case["act"])
        return {"dx": (dz @ w).to(dt), "dw": (dz.T @ s["x"].float()).to(dt), "dbias": dz.sum(0).to(dt)}
    r, c = _rows_cols(case, s["idx"])
    v = s["vals"].float().reshape(-1)
    if op == "decode":
        y = s["bias"].float().repeat(case["rows"], 1)
        return y.index_add_(0, r, w[c] * v[:, None]).to(dt)
    if op == "decode_backward":
        dy = s["dy"].float()
        g = dy[r]
        return {"dvals": (g * w[c]).sum(1).to(dt).reshape(s["vals"].shape), "dw": torch.zeros_like(w).index_add_(0, c, g * v[:, None]).to(dt), "dbias": dy.sum(0).to(dt)}
    dz = s["dvals"].float().reshape(-1) * (v > 0)
    return {"dx": torch.zeros(case["rows"], case["inner"], device=w.device).index_add_(0, r, w[c] * dz[:, None]).to(dt),
            "dw": torch.zeros_like(w).index_add_(0, c, s["x"].float()[r] * dz[:, None]).to(dt),
            "dbias": torch.zeros(case["outer"], device=w.device).index_add_(0, c, dz).to(dt)}


def _own(s):
    import top_selection_prof_gb300 as tk
    case = s["case"]
    op = case["op"]
    if op == "clip_grad_norm":
        norm = tk.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "grads": s["out"]}
    if op == "linear":
        return tk.linear(s["x"], s["w"], s["bias"], act=case["act"], residual=s["residual"])
    if op == "linear_backward":
        dx, dw, dbias = tk.linear_backward(s["dy"], s["x"], s["w"], pre=s["pre"], act=case["act"])
        return {"dx": dx, "dw": dw, "dbias": dbias}
    if op == "decode":
        return tk.decode(s["vals"], s["idx"], s["w"], case["rows"], bias=s["bias"])
    if op == "decode_backward":
        dvals, dw, dbias = tk.decode_backward(s["dy"], s["vals"], s["idx"], s["w"])
        return {"dvals": dvals, "dw": dw, "dbias": dbias}
    dx, dw, dbias = tk.linear_backward_selected(s["dvals"], s["vals"], s["idx"], s["x"], s["w"], act="relu")
    return {"dx": dx, "dw": dw, "dbias": dbias}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip_grad_norm":
        return {"bytes": 2 * size * case["total"] + 4, "flops": 3 * case["total"]}
    m, k, n = case["rows"], case["inner"], case["outer"]
    if case["op"] == "linear":
        return {"bytes": size * (m * k + n * k + n + m * n * (2 if case["residual"] else 1)), "flops": 2 * m * n * k}
    if case["op"] == "linear_backward":
        return {"bytes": size * (m * n * (1 if case["act"] == "none" else 2) + 2 * (m * k + n * k) + n), "flops": 4 * m * n * k}
    places = case["k"] * (m if case["per_row"] else 1)
    touched = min(places, n)
    base = places * (8 + size)
    if case["op"] == "decode":
        return {"bytes": base + size * k * (touched + m + 1), "flops": 2 * places * k}
    if case["op"] == "decode_backward":
        return {"bytes": base + size * (places + k * (touched + n + m + 1)), "flops": 4 * places * k}
    return {"bytes": base + size * (places + k * (touched + n + 2 * m) + n), "flops": 4 * places * k}


def exact(case, seed):
    """The same in 64 bits: selections as a dense matrix with zeros elsewhere, activations from their definitions."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip_grad_norm":
        every = torch.cat([t.double() for t in s["grads"]])
        norm = torch.linalg.vector_norm(every)
        every = every * min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm, "grads": list(every.split([t.numel() for t in s["grads"]]))}
    w = s["w"].double()
    if op in ("linear", "linear_backward"):
        act = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[case["act"]]
        if op == "linear":
            y = act(torch.addmm(s["bias"].double(), s["x"].double(), w.T))
            return y if s["residual"] is None else y + s["residual"].double()
        dz = s["dy"].double()
        if s["pre"] is not None:
            z = s["pre"].double().requires_grad_()
            dz, = torch.autograd.grad(act(z), z, dz)
        return {"dx": dz @ w, "dw": dz.T @ s["x"].double(), "dbias": dz.sum(0)}
    rows, outer = case["rows"], case["outer"]

    def dense(v):
        d = torch.zeros(rows, outer, dtype=torch.float64, device="cuda")
        if case["per_row"]:
            return d.scatter_(1, s["idx"], v.double())
        d.view(-1)[s["idx"]] = v.double()
        return d

    def at(d):
        return d.gather(1, s["idx"]) if case["per_row"] else d.view(-1)[s["idx"]]

    if op == "decode":
        return torch.addmm(s["bias"].double(), dense(s["vals"]), w)
    if op == "decode_backward":
        dy = s["dy"].double()
        return {"dvals": at(dy @ w.T), "dw": dense(s["vals"]).T @ dy, "dbias": dy.sum(0)}
    dz = dense(torch.where(s["vals"] > 0, s["dvals"], torch.zeros_like(s["dvals"])))
    return {"dx": dz @ w, "dw": dz.T @ s["x"].double(), "dbias": dz.sum(0)}
