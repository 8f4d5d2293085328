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
