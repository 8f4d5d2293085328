"""Refusals of the operators of a language model at the C ABI (no kernel is launched here), and what their host code asks the
CUDA runtime for, by the stand-in that the other operators' tests use."""
import ctypes
import os
import random
import subprocess
import sys
import threading

import pytest

from top_selection_prof_gb300 import _lib, build, language

from .test_operators_calls_host import at, events, fake_path, lib  # noqa: F401

VP = ctypes.c_void_p
EINVAL, EUNSUPPORTED = -1, -4
F32, BF16 = 0, 1
NAN, INF = float("nan"), float("inf")


def sample(lib, **kw):  # noqa: F811
    a = dict(logits=at(0), ld=100, dtype=F32, rows=4, n=100, u=at(1), temperature=1.0, temperatures=None, top_k=0, top_ks=None, top_p=1.0,
             top_ps=None, min_p=0.0, min_ps=None, tokens=at(2), logprobs=at(3), stream=None)
    a.update(kw)
    return lib.topk_sample(*a.values())


@pytest.mark.parametrize("bad", [dict(logits=None), dict(u=None), dict(tokens=None), dict(logprobs=None), dict(ld=99), dict(dtype=2), dict(rows=-1),
                                 dict(n=0), dict(temperature=-0.5), dict(temperature=NAN), dict(temperature=INF), dict(top_k=-1), dict(top_p=-0.1),
                                 dict(top_p=1.1), dict(top_p=NAN), dict(min_p=-0.1), dict(min_p=2.0), dict(min_p=NAN), dict(tokens=at(0)),
                                 dict(logprobs=at(1)), dict(tokens=at(3)), dict(temperatures=at(2)), dict(top_ks=at(3))])
def test_sample_refuses(lib, bad):  # noqa: F811
    assert sample(lib, **bad) == EINVAL
    assert not events(lib)


def test_sample_limits(lib):  # noqa: F811
    assert sample(lib, rows=0, logits=None) == 0 and not events(lib)
    assert sample(lib, n=262145, ld=262145) == EUNSUPPORTED
    assert sample(lib, rows=1 << 31) == EUNSUPPORTED
    # numbers that a pointer makes unused are not looked at
    assert sample(lib, temperature=-1.0, temperatures=at(4), top_k=-1, top_ks=at(5), top_p=NAN, top_ps=at(6), min_p=9.0, min_ps=at(7)) == 0
    for dtype in (F32, BF16):
        for rows, n in ((1, 1), (1, 262144), (500, 131072), (100_000, 50)):
            assert sample(lib, rows=rows, n=n, ld=n, dtype=dtype) == 0
    assert all(e[0] == "launch" for e in events(lib))


def dispatch(lib, **kw):  # noqa: F811
    a = dict(x=at(0), ldx=64, idx=at(1), dtype=F32, tokens=4000, k=2, experts=16, d=64, xs=at(2), place=at(3), offsets=at(4), stream=None)
    a.update(kw)
    return lib.topk_dispatch(*a.values())


@pytest.mark.parametrize("bad", [dict(x=None), dict(idx=None), dict(xs=None), dict(place=None), dict(offsets=None), dict(ldx=63), dict(dtype=7),
                                 dict(tokens=-1), dict(k=0), dict(experts=0), dict(d=0), dict(xs=at(0)), dict(place=at(1)), dict(offsets=at(2))])
def test_dispatch_refuses(lib, bad):  # noqa: F811
    assert dispatch(lib, **bad) == EINVAL


def test_dispatch_limits(lib):  # noqa: F811
    assert dispatch(lib, experts=4097) == EUNSUPPORTED
    assert dispatch(lib, tokens=1 << 28, k=2) == EUNSUPPORTED
    assert dispatch(lib, tokens=1 << 31) == EUNSUPPORTED
    room = (ctypes.c_int64 * 17)(7)
    assert dispatch(lib, tokens=0, x=None, offsets=ctypes.addressof(room)) == 0 and room[0] == 0
    assert dispatch(lib, experts=4096) == 0 and dispatch(lib, tokens=3, experts=4096) == 0


def combine(lib, **kw):  # noqa: F811
    a = dict(ys=at(0), ldys=64, rows=900, place=at(1), weights=at(2), dtype=BF16, tokens=300, k=3, d=64, y=at(3), stream=None)
    a.update(kw)
    return lib.topk_combine(*a.values())


@pytest.mark.parametrize("bad", [dict(ys=None), dict(place=None), dict(y=None), dict(ldys=63), dict(dtype=-1), dict(tokens=-1), dict(k=0), dict(d=0),
                                 dict(rows=-1), dict(y=at(0)), dict(y=at(1)), dict(y=at(2))])
def test_combine_refuses(lib, bad):  # noqa: F811
    assert combine(lib, **bad) == EINVAL


def test_combine_limits(lib):  # noqa: F811
    assert combine(lib, tokens=0, y=None) == 0 and combine(lib, rows=0, ys=None) == 0 and combine(lib, weights=None) == 0
    assert combine(lib, rows=1 << 29) == EUNSUPPORTED and combine(lib, tokens=1 << 29, k=1) == EUNSUPPORTED


def combine_backward(lib, **kw):  # noqa: F811
    a = dict(dy=at(0), lddy=64, ys=at(1), ldys=64, rows=900, place=at(2), weights=at(3), dtype=F32, tokens=300, k=3, d=64, dys=at(4), dweights=at(5),
             stream=None)
    a.update(kw)
    return lib.topk_combine_backward(*a.values())


@pytest.mark.parametrize("bad", [dict(dy=None), dict(lddy=63), dict(ys=None), dict(ldys=63), dict(place=None), dict(dtype=3), dict(rows=-1), dict(k=0),
                                 dict(dys=at(0)), dict(dys=at(1)), dict(dweights=at(2)), dict(dweights=at(3)), dict(dweights=at(4))])
def test_combine_backward_refuses(lib, bad):  # noqa: F811
    assert combine_backward(lib, **bad) == EINVAL


def test_combine_backward_needs_only_what_it_reads(lib):  # noqa: F811
    assert combine_backward(lib, dweights=None, ys=None) == 0 and combine_backward(lib, dys=None, dweights=None, dy=None) == 0
    events(lib)
    room = (ctypes.c_float * (900 * 64))(*[1.0] * 3)
    assert combine_backward(lib, tokens=0, dys=ctypes.addressof(room)) == 0 and not any(room[:3])
    assert [e[0] for e in events(lib)] == ["memset"]
    # no rows to write: the weights' gradients alone
    assert combine_backward(lib, rows=0, ys=None) == 0
    assert [e[0] for e in events(lib) if e[0] == "launch"] == ["launch"]
    assert combine_backward(lib, d=(1 << 30) + 1, lddy=1 << 31, ldys=1 << 31) == EUNSUPPORTED


def view(p, batch, head, row=0):
    return None if p is None else ctypes.byref(_lib.TopkView(p.value if isinstance(p, VP) else p, batch, head, row))


B, H, N, D = 3, 4, 256, 64
DENSE, FLAT = (H * N * D, N * D, D), (H * N, N)


def evict(lib, **kw):  # noqa: F811
    a = dict(keys=view(at(0), *DENSE), values=view(at(1), *DENSE), score=view(at(2), *FLAT), lengths=at(3), weights=view(at(4), 2 * H * N, N, N),
             wdtype=F32, group=2, queries=1, dtype=BF16, batch=B, heads=H, capacity=N, kd=D, vd=D, keep=64, recent=8, ok=at(5), ov=at(6), osc=at(7),
             okept=at(8), ol=at(9), stream=None)
    a.update(kw)
    return lib.topk_evict(*a.values())


@pytest.mark.parametrize("bad", [dict(keys=None), dict(values=None), dict(score=None), dict(lengths=None), dict(ok=None), dict(ov=None), dict(osc=None),
                                 dict(okept=None), dict(ol=None), dict(wdtype=5), dict(group=0), dict(queries=-1), dict(dtype=2), dict(batch=-1),
                                 dict(heads=0), dict(capacity=0), dict(kd=0), dict(vd=0), dict(keep=0), dict(recent=-1), dict(recent=65),
                                 dict(ok=at(0)), dict(ov=at(1)), dict(osc=at(2)), dict(okept=at(3)), dict(ol=at(4)), dict(ok=at(6)),
                                 dict(keys=view(at(0), -1, N * D, D)), dict(weights=view(at(4), 2 * H * N, N, -N))])
def test_evict_refuses(lib, bad):  # noqa: F811
    assert evict(lib, **bad) == EINVAL
    assert not events(lib)


def test_evict_limits(lib):  # noqa: F811
    assert evict(lib, batch=0, keys=None) == 0 and evict(lib, weights=None, wdtype=9, group=0) == 0
    assert evict(lib, capacity=1 << 31) == EUNSUPPORTED and evict(lib, keep=1 << 31) == EUNSUPPORTED and evict(lib, batch=1 << 30) == EUNSUPPORTED
    assert evict(lib, kd=(1 << 20) + 1) == EUNSUPPORTED
    events(lib)
    assert evict(lib, wdtype=BF16) == 0


def replace(lib, **kw):  # noqa: F811
    a = dict(keys=view(at(0), *DENSE), values=view(at(1), *DENSE), score=view(at(2), *FLAT), positions=view(at(3), *FLAT), lengths=at(4),
             key=view(at(5), H * D, D), value=view(at(6), H * D, D), weights=view(at(7), H * N, N, N), wdtype=F32, group=1, queries=1, dtype=F32,
             batch=B, heads=H, capacity=N, kd=D, vd=D, recent=8, slots=at(8), stream=None)
    a.update(kw)
    return lib.topk_replace(*a.values())


@pytest.mark.parametrize("bad", [dict(keys=None), dict(values=None), dict(score=None), dict(positions=None), dict(lengths=None), dict(key=None),
                                 dict(value=None), dict(slots=None), dict(wdtype=3), dict(group=0), dict(dtype=4), dict(batch=-1), dict(heads=0),
                                 dict(capacity=0), dict(kd=0), dict(vd=0), dict(recent=-1), dict(recent=N), dict(keys=view(at(1), *DENSE)),
                                 dict(keys=view(at(0), 0, N * D, D)), dict(score=view(at(2), N, N)), dict(positions=view(at(3), H * N, N - 1)),
                                 dict(slots=at(4)), dict(slots=at(2)), dict(key=view(at(0), H * D, D)), dict(weights=view(at(2), H * N, N, N)),
                                 dict(values=view(VP(at(0).value + 4 * (D - 1)), *DENSE))])
def test_replace_refuses(lib, bad):  # noqa: F811
    assert replace(lib, **bad) == EINVAL
    assert not events(lib)


def test_replace_takes_keys_and_values_of_one_buffer(lib):  # noqa: F811
    # rows of a key and a value side by side; positions before heads
    by = (N * H * 2 * D, 2 * D, H * 2 * D)
    assert replace(lib, keys=view(at(0), *by), values=view(VP(at(0).value + 4 * D), *by)) == 0
    assert replace(lib, keys=view(at(0), *by), values=view(VP(at(0).value + 4 * D - 4), *by)) == EINVAL
    assert replace(lib, keys=view(at(0), *by), values=view(VP(at(0).value + 4 * D + 4), *by)) == EINVAL
    assert replace(lib, weights=None) == 0 and replace(lib, batch=0, keys=None) == 0


@pytest.mark.parametrize("first", range(4))
def test_keys_and_values_stacked_along_any_dimension(lib, first):  # noqa: F811
    # (batch, heads, capacity) with the two caches side by side before the first, second, ... of them, or in each row
    n, by, step = [B, H, N], [0, 0, 0], D
    for d in (3, 2, 1, 0):
        if d < 3:
            by[d], step = step, step * n[d]
        if d == first:
            apart, step = step, step * 2
    both = VP(at(0).value + 4 * apart)
    assert replace(lib, keys=view(at(0), *by), values=view(both, *by)) == 0
    assert replace(lib, values=view(at(0), *by), keys=view(both, *by)) == 0
    for off in (-4, 4):
        assert replace(lib, keys=view(at(0), *by), values=view(VP(both.value + off), *by)) == (0 if first == 0 and off > 0 else EINVAL)


@pytest.mark.parametrize("seed", range(40))
def test_caches_that_meet_are_refused_and_no_others(lib, seed):  # noqa: F811
    r = random.Random(seed)
    n = [r.choice([1, 2, 3, 5]) for _ in range(3)]
    dims = [r.choice([1, 3, 8]), r.choice([1, 3, 8])]
    order, by, step = r.sample(range(3), 3), [0, 0, 0], max(dims) * r.choice([1, 2]) + r.randrange(3)
    for d in order:
        by[d], step = step, step * n[d] + r.choice([0, 0, 5, step])
    for _ in range(60):
        off = r.randrange(-step - 5, step + 5)
        bytes_at = [{4 * (base + i * by[0] + j * by[1] + k * by[2] + c) for i in range(n[0]) for j in range(n[1]) for k in range(n[2]) for c in range(dim)}
                    for base, dim in ((0, dims[0]), (off, dims[1]))]
        got = replace(lib, keys=view(at(0), *by), values=view(VP(at(0).value + 4 * off), *by), score=view(at(2), n[1] * n[2], n[2]),
                      positions=view(at(3), n[1] * n[2], n[2]), key=view(at(5), 64, 8), value=view(at(6), 64, 8), weights=None, batch=n[0], heads=n[1],
                      capacity=n[2], kd=dims[0], vd=dims[1], recent=0)
        assert got == (EINVAL if bytes_at[0] & bytes_at[1] else 0), (n, by, dims, off)


def test_weights_of_one_row_repeated_are_bounded(lib):  # noqa: F811
    for call in (evict, replace):
        assert call(lib, weights=view(at(9 if call is replace else 14), 0, 0, 0), group=1 << 15, queries=(1 << 15) + 1) == EUNSUPPORTED
        assert call(lib, weights=view(at(9 if call is replace else 14), 0, 0, 0), group=1 << 15, queries=1 << 15) == 0
    events(lib)


CHAINS = [dispatch, combine_backward, evict]


@pytest.mark.parametrize("call", CHAINS, ids=lambda c: c.__name__)
def test_threads_on_one_stream_do_not_mix_their_launches(lib, call):  # noqa: F811
    assert call(lib) == 0
    chain = sum(e[0] == "launch" for e in events(lib))
    assert chain > 1
    lib.fake_set_launch_us(200)
    failed = []

    def work():
        for _ in range(6):
            if call(lib) != 0:
                failed.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lib.fake_set_launch_us(0)
    who = [e[1] for e in events(lib) if e[0] == "launch"]
    assert not failed and len(who) == 4 * 6 * chain
    assert all(len(set(who[i:i + chain])) == 1 for i in range(0, len(who), chain))


@pytest.mark.parametrize("call", CHAINS, ids=lambda c: c.__name__)
@pytest.mark.parametrize("before", [False, True])
def test_captured_calls_use_memory_of_their_graph(lib, call, before):  # noqa: F811
    stream = 64
    if before:
        assert call(lib, stream=stream) == 0
        events(lib)
    lib.fake_set_capturing(stream, 1)
    for _ in range(2):
        assert call(lib, stream=stream) == 0
        log = [e for e in events(lib) if e[3] == stream]
        made, freed = ([e[4] for e in log if e[0] == kind] for kind in ("malloc", "free"))
        assert len(made) == 1 and made == freed and log[0][0] == "malloc" and log[-1][0] == "free"
    lib.fake_set_capturing(stream, 0)
    assert call(lib, stream=stream) == 0
    log = events(lib)
    assert not any(e[0] == "free" for e in log) and any(e[0] == "malloc" for e in log) != before


@pytest.mark.parametrize("call", [sample, dispatch, combine, combine_backward, evict, replace], ids=lambda c: c.__name__)
def test_a_second_device_is_set_up_like_the_first(lib, call):  # noqa: F811
    launches = []
    for device in (0, 1, 0):
        lib.fake_set_device(device)
        for dtype in (F32, BF16):
            assert call(lib, dtype=dtype) == 0
        log = events(lib)
        assert {e[2] for e in log} == {device}
        launches.append([e[4] for e in log if e[0] == "launch"])
    assert launches[0] == launches[1] == launches[2] and launches[0]
    lib.fake_set_device(0)


# ---- the build ----------------------------------------------------------------------
@pytest.fixture
def tools(tmp_path, monkeypatch):
    """build() with compilers that only write their output, and fail for commands with a word of `fails`; the commands."""
    fails, ran = [], []

    def run(cmd, **kw):
        ran.append(cmd)
        bad = any(word in part for word in fails for part in cmd)
        if not bad:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("made")
        return subprocess.CompletedProcess(cmd, int(bad), "", "no header" if bad else "")

    monkeypatch.setattr(build.subprocess, "run", run)
    for name, at in (("LIB", "libtopk_gb300.so"), ("CALLS", "_language_calls.so"), ("BUILD", "objects")):
        monkeypatch.setattr(build, name, str(tmp_path / at))
    return fails, ran


def test_the_library_is_built_whatever_becomes_of_the_module(tools, monkeypatch, capsys):
    fails, ran = tools
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.CALLS)
    os.remove(build.LIB)
    fails.append("language_calls.cpp")
    with pytest.raises(RuntimeError, match="no header"):
        build.build()
    assert os.path.exists(build.LIB)
    # without torch: no module (a stale one is linked to another library), and no error
    os.remove(build.LIB)
    monkeypatch.setitem(sys.modules, "torch", None)
    del ran[:]
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS) and not any("language_calls" in part for cmd in ran for part in cmd)
    assert "torch cannot be imported" in capsys.readouterr().err


def test_a_module_that_cannot_be_loaded_says_why(monkeypatch, tmp_path):
    monkeypatch.setattr(_lib, "get", lambda: None)
    monkeypatch.setattr(language, "_module", None)
    monkeypatch.setitem(sys.modules, "top_selection_prof_gb300._language_calls", None)
    monkeypatch.delattr("top_selection_prof_gb300._language_calls", raising=False)
    for at, why in ((__file__, "another torch"), (str(tmp_path / "none.so"), "not built")):
        monkeypatch.setattr(language, "CALLS_PATH", at)
        with pytest.raises(RuntimeError, match=why):
            language._calls()
