"""The operators on the GPU as programs call them: from several threads, under capture, on streams of their own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tk():
    import top_selection_prof_gb300 as m
    return m


def normals(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def step(tk, seed, rows, stream=None):
    """A product by parts, a selection, the sums over it and a norm: everything that keeps scratch on its stream."""
    x, w = normals((rows, 64), torch.float32, seed), normals((2048, 64), torch.float32, seed + 1, 0.125)

    def run():
        a = tk.linear(x, w, act="relu", stream=stream)
        v, i = tk.select_global(a, rows * 8, stream=stream)
        y = tk.decode(v, i, w, rows, stream=stream)
        dv, dw, db = tk.decode_backward(y, v, i, w, stream=stream)
        dx, dwe, dbe = tk.linear_backward(a, x, w, pre=a, act="relu", stream=stream)
        return [a, v, i, y, dv, dw, db, dx, dwe, dbe, tk.grad_norm([dw] * 60 + [dwe], stream=stream)]

    return run


def test_threads_on_one_stream(tk):
    """Each thread's results are what they are alone."""
    runs = [step(tk, 10 * t, 100 + 150 * t) for t in range(4)]
    alone = [r() for r in runs]
    torch.cuda.synchronize()
    wrong = []

    def work(t):
        for _ in range(15):
            got = runs[t]()
            wrong.extend(t for p, q in zip(got, alone[t]) if not torch.equal(p, q))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def operators(tk, s):
    """Every operator that keeps scratch or words, on the tensors of s."""
    y, pre = tk.linear(s["x"], s["w"], act="gelu", save_pre=True)
    dx, dw, db = tk.linear_backward(s["dy"], s["x"], s["w"], pre=pre, act="gelu")
    z = tk.decode(s["v"], s["i"], s["w"], s["x"].shape[0])
    dv, dd, _ = tk.decode_backward(z, s["v"], s["i"], s["w"])
    sx, sw, _ = tk.linear_backward_selected(dv, s["v"], s["i"], s["x"], s["w"])
    few = tk.linear(s["x"][:3], s["w"])
    norm = tk.grad_norm([dw, dd, sw] * 20)
    return [y, pre, dx, dw, db, z, dv, dd, sx, sw, few, norm]


def inputs(dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rows, inner, outer = 300, 96, 2000
    i = torch.randperm(rows * outer, generator=g)[:4000]
    i[:300] = torch.arange(300) * outer + 7      # a long column
    s = dict(x=(rows, inner), w=(outer, inner), dy=(rows, outer), v=(4000,))
    return {**{k: torch.randn(z, generator=g).to(dtype).cuda() for k, z in s.items()}, "i": i.cuda()}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured_calls_replay(tk, dtype):
    """A graph of the operators, captured before anything ran on its stream, gives what the calls give: with other inputs, after
    an input that was not finite, beside another graph of the same stream and with calls in between that grow their scratch."""
    s, other = inputs(dtype, 1), inputs(dtype, 2)
    side = torch.cuda.Stream()
    graphs = []
    for state in (s, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = operators(tk, state)
        graphs.append((g, out, state))
    for seed in (3, 4, 5):
        new = inputs(dtype, seed)
        if seed == 4:
            new["x"][5, 7] = torch.inf
        for g, out, state in graphs:
            for k in state:
                state[k].copy_(new[k])
            g.replay()
        big = normals((700, 4096), dtype, seed), normals((600, 4096), dtype, seed + 1)
        with torch.cuda.stream(side):
            tk.linear(*big)
        want = operators(tk, new)
        torch.cuda.synchronize()
        for _, out, _ in graphs:
            for p, q in zip(out, want):
                assert torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0)) and torch.equal(p.isnan(), q.isnan())


def test_captured_product_takes_the_tensor_cores_again(tk):
    """An input that is not finite sends an f32 product to the CUDA cores in the replays that see it, not in those after."""
    x, w = normals((2048, 2048), torch.float32, 1), normals((2048, 2048), torch.float32, 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            y = tk.linear(x, w)

    def time():
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        g.replay()
        a.record()
        for _ in range(5):
            g.replay()
        b.record()
        b.synchronize()
        return a.elapsed_time(b)

    before = time()
    first = y.clone()
    keep = x[3, 3].clone()
    x[3, 3] = torch.nan
    g.replay()
    torch.cuda.synchronize()
    assert y[3].isnan().all() and y[4].isfinite().all()
    x[3, 3] = keep
    after = time()
    assert torch.equal(y, first)     # (the CUDA cores' sums have other bits)
    assert after < 3 * before


# paths of the selection: the whole tensor (bins, grid refinement), one long row, rows by blocks, rows by clusters
@pytest.mark.parametrize("rows,n,k,whole", [(512, 16384, 4096, True), (1, 1 << 22, 64, False), (300, 4096, 32, False),
                                            (4, 100_000, 2000, False)])
def test_captured_selection_replays(tk, rows, n, k, whole):
    """A captured selection gives what the call gives, with other inputs, replay after replay."""
    x = normals((rows, n), torch.float32, 1)
    call = tk.select_global if whole else tk.select
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v, i = call(x, k)
    for seed in range(2, 7):
        x.copy_(normals((rows, n), torch.float32, seed))
        g.replay()
        want = call(x, k)
        assert torch.equal(v, want[0]) and torch.equal(i, want[1])


def test_results_over_their_inputs_are_refused(tk):
    x, w = torch.ones(50, 64, device="cuda"), torch.ones(64, 64, device="cuda")
    both = torch.ones(50, 128, device="cuda")
    for call in (lambda: tk.linear(x, w, out=x), lambda: tk.linear(x, w, out=w[:50]),
                 lambda: tk.linear(x, w, residual=both[:, :64], out=both[:, 32:96])):
        with pytest.raises(tk.TopkError) as err:
            call()
        assert err.value.status == -1
    assert torch.equal(tk.linear(both[:, :64], w, out=both[:, 64:]), torch.full((50, 64), 64.0, device="cuda"))
    assert torch.equal(both[:, :64], x) and torch.equal(w, torch.ones_like(w))


LONG = 100_000_000   # cycles, some 50 ms


def test_outputs_on_another_stream_do_not_take_memory_in_use(tk):
    """An output written by a side stream at once is not in memory that the current stream still has to read."""
    side = torch.cuda.Stream()
    x, w = torch.ones(300, 64, device="cuda"), torch.ones(512, 64, device="cuda")
    v, i = torch.ones(900, device="cuda"), torch.arange(900, device="cuda") * 7
    torch.cuda.synchronize()
    calls = {(300, 512): lambda: tk.linear(x, w, stream=side), (300, 64): lambda: tk.decode(v, i, w, 300, stream=side),
             (512, 64): lambda: tk.decode_backward(x, v, i, w, stream=side)[1], (4096,): lambda: tk.select_global(x, 4096, stream=side)[0]}
    for shape, call in calls.items():
        t = torch.full(shape, 5.0, device="cuda")
        torch.cuda._sleep(LONG)
        keep = t.clone()       # waits for the sleep
        del t                  # its memory goes back to the current stream's pool
        out = call()
        torch.cuda.synchronize()
        assert out.shape == shape and bool((keep == 5.0).all())


def test_outputs_and_inputs_live_as_long_as_both_streams_use_them(tk):
    side = torch.cuda.Stream()
    w = torch.ones(512, 64, device="cuda")
    x = torch.ones(300, 64, device="cuda")
    torch.cuda.synchronize()
    y = tk.linear(x, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    keep = y.clone()           # on the current stream, later
    del y
    again = [tk.linear(x, w[:512], bias=w[:, 0].contiguous(), stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert bool((keep == 64.0).all()) and all(bool((a == 65.0).all()) for a in again)
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    y = tk.linear(x, w, stream=side)     # reads x after the sleep
    v, _ = tk.select_global(x, 100, stream=side)
    del x
    other = [torch.full((300, 64), 9.0, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert bool((y == 64.0).all()) and bool((v == 1.0).all()) and len(other) == 3
