"""Arguments that the products of rows, the row norm and the activation's
gradient refuse, and the sizes of their workspaces, on the CPU: nothing
reaches a device."""
import ctypes

import pytest

import submanifold_sparse_convolution_device_amd as sp
from test_attention_abi_host import FAKE, _status

BAD, UNSUPPORTED = "SPCONV_ERR_INVALID_ARG", "SPCONV_ERR_UNSUPPORTED"


def _linear(**change):
    a = dict(x=FAKE, weight=2 * FAKE, cu=0, x_row_stride=64, rows=16, groups=1, c_in=64, c_out=32, activation=0, dtype=1)
    a.update(change)
    return sp.spconv_linear(**a)


def _epilogue(**change):
    a = dict(bias=4 * FAKE, residual=5 * FAKE, out=6 * FAKE, pre=0, residual_row_stride=32, out_row_stride=32, pre_row_stride=0)
    a.update(change)
    return sp.spconv_linear_epilogue(**a)


def _gradients(**change):
    a = dict(grad_out=7 * FAKE, before=0, grad_x=8 * FAKE, grad_weight=16 * FAKE, grad_bias=24 * FAKE, grad_out_row_stride=32,
             before_row_stride=64, grad_x_row_stride=64)
    a.update(change)
    return sp.spconv_linear_gradients(**a)


def _norm(**change):
    a = dict(x=FAKE, residual=8 * FAKE, weight=16 * FAKE, x_row_stride=64, residual_row_stride=64, rows=16, channels=64, eps=1e-6, dtype=1)
    a.update(change)
    return sp.spconv_add_norm(**a)


def _norm_gradients(**change):
    a = dict(grad_h=24 * FAKE, grad_y=32 * FAKE, grad=40 * FAKE, grad_weight=48 * FAKE, grad_h_row_stride=64, grad_y_row_stride=64,
             grad_row_stride=64)
    a.update(change)
    return sp.spconv_add_norm_gradients(**a)


@pytest.mark.parametrize("change", [
    dict(x=0), dict(x=FAKE + 8), dict(weight=0), dict(weight=2 * FAKE + 4), dict(x_row_stride=63), dict(x_row_stride=1 << 22),
    dict(rows=-1), dict(rows=(1 << 30) + 1), dict(c_in=0), dict(c_out=0), dict(c_in=1 << 19), dict(c_out=1 << 19), dict(groups=0),
    dict(groups=2), dict(groups=1 << 16, cu=FAKE * 30), dict(cu=30 * FAKE + 2), dict(activation=4), dict(activation=-1),
    dict(rows=1 << 30, x_row_stride=1 << 12, c_in=1 << 12, c_out=1 << 18)])
def test_linear_sizes(change):
    assert _status(sp.spconv_linear_forward, _linear(**change), _epilogue(), 0) == BAD
    assert _status(sp.spconv_linear_backward, _linear(**change), _gradients(), 0) == BAD


def test_linear_types_and_nulls():
    assert _status(sp.spconv_linear_forward, _linear(dtype=3), _epilogue(), 0) == UNSUPPORTED
    assert _status(sp.spconv_linear_backward, _linear(dtype=-1), _gradients(), 0) == UNSUPPORTED
    L, a = sp.lib(), _linear()
    for f in (L.spconv_linear_forward, L.spconv_linear_backward):
        assert sp.STATUS[f(None, None, None)] == sp.STATUS[f(ctypes.byref(a), None, None)] == BAD


@pytest.mark.parametrize("change", [
    dict(out=0), dict(out=6 * FAKE + 1), dict(out_row_stride=31), dict(residual_row_stride=16), dict(residual=5 * FAKE + 1), dict(bias=1),
    dict(pre=7 * FAKE, pre_row_stride=8), dict(out=FAKE), dict(out=2 * FAKE), dict(out=4 * FAKE), dict(out=5 * FAKE + 2),
    dict(out=5 * FAKE, out_row_stride=40), dict(pre=6 * FAKE, pre_row_stride=32), dict(pre=5 * FAKE, pre_row_stride=32)])
def test_linear_epilogue(change):
    assert _status(sp.spconv_linear_forward, _linear(), _epilogue(**change), 0) == BAD


@pytest.mark.parametrize("change,args", [
    (dict(grad_out=0), {}), (dict(grad_out=7 * FAKE + 8), {}), (dict(grad_out_row_stride=36), {}), (dict(grad_out_row_stride=24), {}),
    (dict(before=9 * FAKE), {}), (dict(before=9 * FAKE, before_row_stride=8), dict(activation=3)), (dict(grad_weight=0), {}),
    (dict(grad_x_row_stride=32), {}), (dict(grad_x=FAKE), {}), (dict(grad_x=7 * FAKE), {}), (dict(grad_x=16 * FAKE), {}),
    (dict(grad_weight=2 * FAKE), {}), (dict(grad_weight=16 * FAKE + 2), {}), (dict(grad_bias=16 * FAKE + 64), {}),
    (dict(grad_bias=24 * FAKE + 1), {}), (dict(before=8 * FAKE), dict(activation=1))])
def test_linear_gradients(change, args):
    assert _status(sp.spconv_linear_backward, _linear(**args), _gradients(**change), 0) == BAD


def test_linear_workspaces():
    # whole pieces and enough tiles: the forward needs none
    assert sp.spconv_linear_workspace(_linear(rows=100000))[0] == 0
    # odd lengths are laid out: x, and the weights
    f, b = sp.spconv_linear_workspace(_linear(rows=100000, c_in=33, x_row_stride=33, c_out=7))
    assert f >= 100000 * 40 * 2 and b >= 100000 * (40 + 8) * 2
    # few rows over a long contraction go by parts
    f, _ = sp.spconv_linear_workspace(_linear(rows=4, c_in=4096, x_row_stride=4096))
    assert f > 0
    none = dict(x=0, weight=0)
    assert sp.spconv_linear_workspace(_linear(rows=4, c_in=4096, x_row_stride=4096, **none))[0] == f
    assert sp.spconv_linear_workspace(_linear(rows=0))[0] == 0
    assert sp.lib().spconv_linear_workspace(ctypes.byref(_linear()), None, None) == 0
    assert _status(sp.spconv_linear_workspace, _linear(c_in=0)) == BAD
    assert sp.STATUS[sp.lib().spconv_linear_workspace(None, None, None)] == BAD


@pytest.mark.parametrize("place,short", [(0, 0), (1 << 20, 1), ((1 << 20) + 8, 0), (FAKE, 0), (6 * FAKE, 0)])
def test_linear_refused_workspaces(place, short):
    """NULL, too small by a byte, misaligned, over an input and over the output."""
    a = _linear(rows=4, c_in=4096, x_row_stride=4096, weight=1 << 24)
    need = sp.spconv_linear_workspace(a)[0]
    e = _epilogue(out=1 << 28 if place != 6 * FAKE else 1 << 18)
    assert _status(sp.spconv_linear_forward_noalloc, a, e, place if place != 6 * FAKE else 1 << 18, need - short, 0) == BAD
    a = _linear(rows=5000, c_in=33, x_row_stride=33, x=1 << 26)
    need = sp.spconv_linear_workspace(a)[1]
    g = _gradients(grad_x_row_stride=33, grad_out=1 << 27, grad_x=1 << 28, grad_weight=1 << 29, grad_bias=1 << 30)
    assert _status(sp.spconv_linear_backward_noalloc, a, g, 1 << 26 if place == FAKE else 1 << 28 if place == 6 * FAKE else place,
                   need - short, 0) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(x=0), BAD), (dict(x=FAKE + 8), BAD), (dict(x_row_stride=60), BAD), (dict(x_row_stride=68), BAD), (dict(x_row_stride=1 << 24), BAD),
    (dict(residual=8 * FAKE + 2), BAD), (dict(residual_row_stride=0), BAD), (dict(weight=0), BAD), (dict(weight=16 * FAKE + 8), BAD),
    (dict(rows=-1), BAD), (dict(rows=(1 << 30) + 1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(channels=0), UNSUPPORTED), (dict(channels=12), UNSUPPORTED), (dict(channels=16392), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED),
    (dict(rows=1 << 30, channels=16384, x_row_stride=16384), BAD)])
def test_add_norm_arguments(change, status):
    assert _status(sp.spconv_add_norm_forward, _norm(**change), 50 * FAKE, 64, 60 * FAKE, 64, 0) == status
    if "residual" not in next(iter(change)):
        assert _status(sp.spconv_add_norm_backward, _norm(**change), _norm_gradients(), 0) == status


def test_add_norm_outputs():
    f = sp.spconv_add_norm_forward
    assert _status(f, _norm(), 0, 64, 60 * FAKE, 64, 0) == BAD
    assert _status(f, _norm(), 50 * FAKE, 64, 0, 64, 0) == BAD
    assert _status(f, _norm(), 50 * FAKE, 64, 50 * FAKE, 64, 0) == BAD
    assert _status(f, _norm(), 50 * FAKE, 64, 16 * FAKE, 64, 0) == BAD
    assert _status(f, _norm(), 50 * FAKE + 8, 64, 60 * FAKE, 64, 0) == BAD
    assert _status(f, _norm(), FAKE + 16, 64, 60 * FAKE, 64, 0) == BAD
    assert _status(f, _norm(), FAKE, 72, 60 * FAKE, 64, 0) == BAD
    assert _status(f, _norm(residual=0), 50 * FAKE, 64, 60 * FAKE, 64, 0) == BAD
    b = sp.spconv_add_norm_backward
    for change in (dict(grad_y=0), dict(grad=0), dict(grad=FAKE), dict(grad=16 * FAKE), dict(grad_weight=48 * FAKE + 1), dict(grad_weight=FAKE),
                   dict(grad=24 * FAKE + 16), dict(grad_weight=40 * FAKE), dict(grad_h_row_stride=32), dict(grad_h=24 * FAKE + 4)):
        assert _status(b, _norm(), _norm_gradients(**change), 0) == BAD
    L, a = sp.lib(), _norm()
    assert sp.STATUS[L.spconv_add_norm_forward(None, None, 0, None, 0, None)] == BAD
    assert sp.STATUS[L.spconv_add_norm_backward(ctypes.byref(a), None, None)] == BAD


def test_add_norm_workspace():
    assert sp.spconv_add_norm_workspace(4096) == 512 * sp.spconv_add_norm_workspace(8) > 0
    assert _status(sp.spconv_add_norm_workspace, 12) == UNSUPPORTED
    assert _status(sp.spconv_add_norm_workspace, 16392) == UNSUPPORTED
    assert sp.STATUS[sp.lib().spconv_add_norm_workspace(32, None)] == BAD
    need = sp.spconv_add_norm_workspace(64)
    for place, size in ((0, need), (1 << 22, need - 1), ((1 << 22) + 8, need), (FAKE, need), (40 * FAKE, need)):
        assert _status(sp.spconv_add_norm_backward_noalloc, _norm(), _norm_gradients(), place, size, 0) == BAD


def test_activation_backward_arguments():
    f = sp.spconv_activation_backward
    good = dict(g=FAKE, gs=16, p=8 * FAKE, ps=16, o=16 * FAKE, os=16, rows=8, channels=16, act=3, dtype=1)
    for change in (dict(g=0), dict(g=FAKE + 1), dict(gs=8), dict(p=0), dict(ps=15), dict(o=0), dict(os=1 << 22), dict(rows=-1),
                   dict(channels=0), dict(channels=1 << 19), dict(act=4), dict(act=-1), dict(o=8 * FAKE), dict(o=FAKE + 2),
                   dict(rows=1 << 30, channels=1 << 10, gs=1 << 10, ps=1 << 10, os=1 << 10)):
        assert _status(f, *{**good, **change}.values(), 0) == BAD, change
    assert _status(f, *{**good, "dtype": 3}.values(), 0) == UNSUPPORTED


def test_packed_structs_mirror_the_c_structs():
    for packed, mirror in ((sp._PACK_ADD_NORM, sp.spconv_add_norm), (sp._PACK_ADD_NORM_GRADIENTS, sp.spconv_add_norm_gradients),
                           (sp._PACK_LINEAR, sp.spconv_linear), (sp._PACK_LINEAR_EPILOGUE, sp.spconv_linear_epilogue),
                           (sp._PACK_LINEAR_GRADIENTS, sp.spconv_linear_gradients)):
        assert packed.size == ctypes.sizeof(mirror)
