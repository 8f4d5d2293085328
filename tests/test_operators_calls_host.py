"""What the host code of the operators asks the CUDA runtime for, seen by a stand-in for it (fake_cudart.cpp): no GPU.

The library's own objects are linked with the stand-in, and the C entries are called with addresses that nothing touches.
"""
import ctypes
import os
import re
import subprocess
import threading
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VP = ctypes.c_void_p
F32, BF16 = 0, 1


@pytest.fixture(scope="session")
def fake_path(tmp_path_factory):
    from top_selection_prof_gb300 import build
    objects = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    sources = [os.path.join(build.CSRC, f) for f in os.listdir(build.CSRC)]
    if not all(map(os.path.exists, objects)) or min(map(os.path.getmtime, objects)) < max(map(os.path.getmtime, sources)):
        build.build()
    out = str(tmp_path_factory.mktemp("fake") / "libtopk_fake.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", include, "-o", out,
                    os.path.join(ROOT, "tests", "fake_cudart.cpp"), *objects, "-lpthread", "-Wl,-z,defs,-Bsymbolic"], check=True)
    return out


@pytest.fixture
def lib(fake_path, tmp_path):
    """The library anew for each test: a copy, as one path is loaded once."""
    import shutil
    from top_selection_prof_gb300 import _lib
    path = str(tmp_path / "lib.so")
    shutil.copy(fake_path, path)
    lib = ctypes.CDLL(path)
    lib.fake_take_log.restype = ctypes.c_char_p
    lib.fake_set_capturing.argtypes = [VP, ctypes.c_int]
    real = _lib.get()
    for name in _lib.EXPORTS:
        getattr(lib, name).argtypes = getattr(real, name).argtypes
        getattr(lib, name).restype = getattr(real, name).restype
    return lib


def at(i):
    return VP((i + 1) << 40)   # never touched


def events(lib):
    got = []
    for line in lib.fake_take_log().decode().splitlines():
        m = re.match(r"(\w+) thread=(\d+) device=(\d+) stream=(\d+) (\S+)", line)
        got.append((m[1], int(m[2]), int(m[3]), int(m[4]), m[5]))
    return got


def linear(lib, stream=0, dtype=F32, rows=300, inner=64, outer=512):
    return lib.topk_linear(at(0), inner, at(1), inner, None, None, 0, dtype, rows, inner, outer, 0, at(2), outer, None, 0, stream)


def linear_backward(lib, stream=0, dtype=BF16, rows=300, inner=64, outer=512, act=3):
    return lib.topk_linear_backward(at(0), outer, at(1), inner, at(2), inner, at(3), outer, dtype, rows, inner, outer, act, at(4),
                                    at(5), at(6), stream)


def decode_backward(lib, stream=0, dtype=F32, rows=300, n=2000, d=512, count=5000):
    return lib.topk_decode_backward(at(0), d, at(1), at(2), count, 0, at(3), d, dtype, rows, n, d, at(4), at(5), at(6), stream)


def clip(lib, stream=0, num=700, count=1000):
    ptrs = (VP * num)(*[(i + 1) << 20 for i in range(num)])
    return lib.topk_clip_grad_norm(ptrs, ptrs, (ctypes.c_int64 * num)(*[count] * num), (ctypes.c_int * num)(*[F32] * num), num,
                                   1.0, at(2), stream)


def select(lib, stream=0):
    return lib.topk_select_global(at(0), BF16, 512, 16384, 4096, 1, 1e-3, at(1), at(2), stream)


CALLS = [linear, linear_backward, decode_backward, clip, select]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_threads_on_one_stream_do_not_mix_their_launches(lib, call):
    """A call's launches share scratch: those of another thread's call on the stream may not come between them."""
    assert call(lib) == 0
    chain = sum(e[0] == "launch" for e in events(lib))
    assert chain > 1
    assert call(lib) == 0            # (the first call also made its scratch)
    assert sum(e[0] == "launch" for e in events(lib)) == chain
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


def test_scratch_grown_by_one_thread_is_not_another_calls(lib):
    """A larger call releases the block in stream order: after the whole chain that uses it, not in its middle."""
    assert linear(lib, inner=2048) == 0
    chain = sum(e[0] == "launch" for e in events(lib))
    lib.fake_set_launch_us(300)
    small = threading.Thread(target=lambda: [linear(lib, inner=2048) for _ in range(8)])
    # (out of step with the other's launches)
    large = threading.Thread(target=lambda: [(time.sleep(0.0004), linear(lib, rows=300 << i, inner=2048)) for i in range(1, 6)])
    small.start(), large.start()
    small.join(), large.join()
    lib.fake_set_launch_us(0)
    done = {}   # launches of each thread
    log = events(lib)
    assert sum(e[0] == "free" for e in log) >= 3
    for e in log:
        if e[0] == "launch":
            done[e[1]] = done.get(e[1], 0) + 1
        if e[0] == "free":
            assert all(n % chain == 0 for n in done.values())


def test_threads_have_scratch_of_their_own_on_the_per_thread_stream(lib):
    per_thread = 2   # cudaStreamPerThread: one handle, a stream of each thread
    made = []

    def work():
        assert linear(lib, stream=per_thread) == 0
        made.append([e[4] for e in events(lib) if e[0] == "malloc"])

    for _ in range(2):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    assert len(made) == 2 and made[0] and made[1]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
@pytest.mark.parametrize("before", [False, True])
def test_captured_calls_use_memory_of_their_graph(lib, call, before):
    """Captured: scratch that is made and released in the graph, words at zero in each replay, and nothing of it kept."""
    stream = 64
    if before:
        assert call(lib, stream=stream) == 0
        outside = {e[4] for e in events(lib) if e[0] == "malloc"}
    lib.fake_set_capturing(stream, 1)
    for _ in range(2):
        assert call(lib, stream=stream) == 0
        log = [e for e in events(lib) if e[3] == stream]
        made, freed = ([e[4] for e in log if e[0] == kind] for kind in ("malloc", "free"))
        assert len(made) == 1 and made == freed
        assert log[0][0] == "malloc" and log[-1][0] == "free"     # before the first launch, after the last
    lib.fake_set_capturing(stream, 0)
    assert call(lib, stream=stream) == 0
    log = events(lib)
    assert not any(e[0] == "free" for e in log)
    assert any(e[0] == "malloc" for e in log) != before          # its own block, made outside the graph


@pytest.mark.parametrize("call", [linear, linear_backward, decode_backward, clip], ids=lambda c: c.__name__)
def test_a_second_device_is_set_up_like_the_first(lib, call):
    """What a kernel needs before its launch (its shared memory) belongs to a device, not to the process."""
    launches = []
    for device in (0, 1, 0):
        lib.fake_set_device(device)
        for dtype in (F32, BF16) if call is not clip else (None,):
            assert (call(lib) if call is clip else call(lib, dtype=dtype)) == 0
        log = events(lib)
        assert {e[2] for e in log} == {device}
        launches.append([e[4] for e in log if e[0] == "launch"])
    assert launches[0] == launches[1] == launches[2]
    lib.fake_set_device(0)


def span(p, rows, cols, ld):
    return {p + r * ld + c for r in range(rows) for c in range(cols)}


def test_outputs_that_overlap_are_refused(lib):
    """linear's y and the other tensors at every place of a small buffer, against the sets of bytes they have."""
    base, rows, inner, outer = 1 << 20, 3, 2, 2
    seen = set()
    for ldx in (2, 5):
        for ldy in (2, 5):
            for shift in range(-16, 17):
                x = span(base, rows, 4 * inner, 4 * ldx)
                y = span(base + 4 * shift, rows, 4 * outer, 4 * ldy)
                rc = lib.topk_linear(base, ldx, at(1), inner, None, None, 0, F32, rows, inner, outer, 0, base + 4 * shift, ldy, None,
                                     0, None)
                # (rows of unequal distance: any two ranges that meet)
                met = bool(x & y) if ldx == ldy else max(x) >= min(y) and max(y) >= min(x)
                assert rc == (-1 if met else 0), (ldx, ldy, shift)
                seen.add((ldx == ldy, met))
    assert len(seen) == 4
    b = at(0).value
    for refused, kw in ((True, dict(y=b)), (True, dict(y=b + 64)), (False, dict(r=at(2).value)), (True, dict(r=at(2).value + 4)),
                        (True, dict(r=at(2).value, ldr=600)), (True, dict(pre=at(2).value)), (True, dict(pre=b)),
                        (True, dict(r=at(3).value, pre=at(3).value)), (True, dict(bias=at(2).value + 400)), (False, dict(pre=at(3).value)),
                        (True, dict(y=at(1).value - 4))):
        a = dict(bias=None, r=None, ldr=512, y=at(2).value, pre=None)
        a.update(kw)
        rc = lib.topk_linear(b, 64, at(1), 64, a["bias"], a["r"], a["ldr"], F32, 300, 64, 512, 0, a["y"], 512, a["pre"], 512, None)
        assert rc == (-1 if refused else 0), kw


@pytest.mark.parametrize("i,j", [(4, 0), (4, 2), (4, 3), (5, 1), (6, 0), (5, 4), (6, 5)])
def test_gradients_that_overlap_are_refused(lib, i, j):
    p = [at(k).value for k in range(7)]
    call = lambda: lib.topk_linear_backward(p[0], 512, p[1], 64, p[2], 64, p[3], 512, BF16, 300, 64, 512, 3, p[4], p[5], p[6], None)  # noqa: E731
    assert call() == 0
    p[i] = p[j] + 16
    assert call() == -1


def test_selections_and_norms_that_overlap_are_refused(lib):
    def decode_(y):
        return lib.topk_decode(at(0), at(1), 5, 0, at(2), 8, at(3), F32, 4, 6, 8, y, None)

    def back(dvals, dw):
        return lib.topk_decode_backward(at(0), 8, at(1), at(2), 5, 0, at(3), 8, F32, 4, 6, 8, dvals, dw, at(6), None)

    def selected(dx, db):
        return lib.topk_linear_backward_selected(at(0), at(1), at(2), 5, 0, at(3), 8, at(4), 8, F32, 4, 8, 6, 1, dx, at(6), db, None)

    def clip_(src, dst):
        one = (VP * 1)(src), (VP * 1)(dst), (ctypes.c_int64 * 1)(100), (ctypes.c_int * 1)(F32)
        return lib.topk_clip_grad_norm(*one, 1, 1.0, at(2), None)

    assert decode_(at(4)) == 0 and back(at(4), at(5)) == 0 and selected(at(5), at(7)) == 0
    assert all(decode_(at(i)) == -1 for i in range(4))
    assert all(back(at(i), at(5)) == -1 and back(at(5), at(i)) == -1 for i in (0, 1, 2, 3, 6) if i != 1) and back(at(4), at(4)) == -1
    assert all(selected(at(i), at(7)) == -1 and selected(at(5), at(i)) == -1 for i in (0, 1, 2, 3, 4, 6))
    assert clip_(1 << 20, 1 << 20) == 0 and clip_(1 << 20, (1 << 20) + 400) == 0 and clip_(1 << 20, (1 << 20) + 396) == -1


def test_a_wait_that_ran_out_is_told_once(lib):
    """The status word that a kernel sets when a device wait gives up, written here by the test."""
    stream, timeout, etimeout = 64, 1, -5
    assert lib.topk_last_status(stream) == 0
    assert linear(lib, stream=stream) == 0
    zeroed = [e[4] for e in events(lib) if e[0] == "memset"]
    assert len(zeroed) == 1
    word = ctypes.c_int.from_address(int(zeroed[0], 16))
    assert lib.topk_last_status(stream) == 0
    word.value = timeout
    assert lib.topk_last_status(stream) == etimeout
    assert lib.topk_last_status(stream) == 0 and word.value == 0
