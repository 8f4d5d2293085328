"""Refusals of the operators around the selection at the C ABI (no kernel is launched here)."""
import ctypes
import os

import pytest

VP = ctypes.c_void_p
P = VP(16)   # never dereferenced: the checks come before any launch
EINVAL, EUNSUPPORTED = -1, -4


@pytest.fixture(scope="module")
def lib():
    from top_selection_prof_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from top_selection_prof_gb300 import build
        build.build()
    return _lib.get()


def linear(lib, **kw):
    a = dict(x=P, ldx=8, w=P, ldw=8, bias=None, residual=None, ldr=0, dtype=0, rows=4, inner=8, outer=6, act=0, y=P,
             ldy=6, pre=None, ldp=0)
    a.update(kw)
    return lib.topk_linear(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(y=None), dict(ldx=7), dict(ldw=7), dict(ldy=5),
                                 dict(dtype=2), dict(dtype=-1), dict(rows=-1), dict(inner=0), dict(outer=0),
                                 dict(act=4), dict(act=-1), dict(residual=P, ldr=5), dict(pre=P, ldp=5)])
def test_linear_refuses(lib, bad):
    assert linear(lib, **bad) == EINVAL


def test_linear_no_rows_and_extents(lib):
    assert linear(lib, rows=0, x=None, y=None) == 0
    big = 1 << 31
    assert linear(lib, rows=big) == EUNSUPPORTED
    assert linear(lib, inner=big, ldx=big, ldw=big) == EUNSUPPORTED
    assert linear(lib, outer=big, ldy=big) == EUNSUPPORTED


def linear_backward(lib, **kw):
    a = dict(dy=P, lddy=6, x=P, ldx=8, w=P, ldw=8, pre=P, ldp=6, dtype=1, rows=4, inner=8, outer=6, act=1, dx=P, dw=P,
             dbias=P)
    a.update(kw)
    return lib.topk_linear_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(dy=None), dict(lddy=5), dict(x=None), dict(ldx=7), dict(w=None), dict(ldw=7),
                                 dict(pre=None), dict(ldp=5), dict(dtype=9), dict(rows=-2), dict(inner=0),
                                 dict(outer=-1), dict(act=7)])
def test_linear_backward_refuses(lib, bad):
    assert linear_backward(lib, **bad) == EINVAL


def test_linear_backward_without_outputs(lib):
    assert linear_backward(lib, dx=None, dw=None, dbias=None) == 0
    assert linear_backward(lib, rows=1 << 31) == EUNSUPPORTED


def selected(lib, **kw):
    a = dict(dvals=P, vals=P, idx=P, count=3, per_row=0, x=P, ldx=8, w=P, ldw=8, dtype=0, rows=4, inner=8, outer=6, act=1,
             dx=P, dw=P, dbias=P)
    a.update(kw)
    return lib.topk_linear_backward_selected(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(dvals=None), dict(vals=None), dict(idx=None), dict(count=-1), dict(x=None),
                                 dict(ldx=7), dict(w=None), dict(ldw=7), dict(dtype=2), dict(rows=-1), dict(inner=0),
                                 dict(outer=0), dict(act=2), dict(act=3)])
def test_selected_backward_refuses(lib, bad):
    assert selected(lib, **bad) == EINVAL


def decode(lib, **kw):
    a = dict(vals=P, idx=P, count=3, per_row=0, w=P, ldw=8, bias=None, dtype=0, rows=4, n=6, d=8, y=P)
    a.update(kw)
    return lib.topk_decode(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(vals=None), dict(idx=None), dict(count=-1), dict(w=None), dict(ldw=7), dict(y=None),
                                 dict(dtype=3), dict(rows=-1), dict(n=0), dict(d=0)])
def test_decode_refuses(lib, bad):
    assert decode(lib, **bad) == EINVAL


def test_decode_extents(lib):
    assert decode(lib, rows=0, y=None) == 0
    assert decode(lib, count=1 << 31) == EUNSUPPORTED
    assert decode(lib, per_row=1, count=1 << 20, rows=1 << 12) == EUNSUPPORTED
    assert decode(lib, n=1 << 31) == EUNSUPPORTED


def decode_backward(lib, **kw):
    a = dict(dy=P, lddy=8, vals=P, idx=P, count=3, per_row=0, w=P, ldw=8, dtype=0, rows=4, n=6, d=8, dvals=P, dw=P,
             dbias=P)
    a.update(kw)
    return lib.topk_decode_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(dy=None), dict(lddy=7), dict(vals=None), dict(idx=None), dict(count=-5),
                                 dict(w=None), dict(ldw=7), dict(dtype=5), dict(rows=-1), dict(n=0), dict(d=0)])
def test_decode_backward_refuses(lib, bad):
    assert decode_backward(lib, **bad) == EINVAL


def clip(lib, num=1, ptr=16, out=16, count=5, dtype=0, max_norm=1.0, norm=P):
    arr = (VP * 1)(ptr)
    outs = (VP * 1)(out)
    return lib.topk_clip_grad_norm(arr, outs, (ctypes.c_int64 * 1)(count), (ctypes.c_int * 1)(dtype), num, max_norm, norm,
                                   None)


@pytest.mark.parametrize("bad", [dict(num=-1), dict(ptr=None), dict(out=None), dict(count=-1), dict(dtype=2),
                                 dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None)])
def test_clip_refuses(lib, bad):
    assert clip(lib, **bad) == EINVAL


def test_norm_refuses(lib):
    one = (ctypes.c_int64 * 1)(4), (ctypes.c_int * 1)(0)
    assert lib.topk_grad_norm((VP * 1)(16), *one, 1, None, None) == EINVAL
    assert lib.topk_grad_norm((VP * 1)(None), *one, 1, P, None) == EINVAL
    assert lib.topk_grad_norm(None, *one, 1, P, None) == EINVAL
