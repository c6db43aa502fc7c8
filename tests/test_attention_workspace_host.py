"""The workspaces that callers of attention and of the head norm's gradient
bring: their sizes and refusals, on the CPU."""
import ctypes

import pytest

import submanifold_sparse_convolution_device_amd as sp
from test_attention_abi_host import FAKE, _attention, _norm, _status


def _gradients():
    return sp.spconv_attention_gradients(grad_out=6 * FAKE, grad_out_row_stride=128, grad_out_head_stride=32, grad_q=7 * FAKE,
                                         grad_q_row_stride=128, grad_q_head_stride=32, grad_k=8 * FAKE, grad_k_row_stride=64,
                                         grad_k_head_stride=32, grad_v=9 * FAKE, grad_v_row_stride=64, grad_v_head_stride=32)


def test_sizes():
    # whole short sequences: no parts to join; the gradient keeps two fp32 statistics of each row and head
    f, b = sp.spconv_attention_workspace(_attention(total_q=6400, total_k=6400, batch=640))
    assert f == 0 and 6400 * 4 * 8 <= b < 6400 * 4 * 8 + 4096
    # single queries over long keys go by parts
    f, _ = sp.spconv_attention_workspace(_attention(total_q=8, total_k=80000, batch=8))
    assert f > 0
    # sizes alone: no pointer is looked at
    none = dict.fromkeys(("q", "k", "v", "cu_q", "cu_k"), 0)
    assert sp.spconv_attention_workspace(_attention(total_q=8, total_k=80000, batch=8, **none))[0] == f
    assert sp.spconv_attention_workspace(_attention(total_q=0, total_k=0)) == (0, 0)
    assert sp.spconv_norm_rotary_workspace(128) == 16 * sp.spconv_norm_rotary_workspace(8) > 0
    a = _attention()
    assert sp.lib().spconv_attention_workspace(ctypes.byref(a), None, None) == 0


def test_parts_are_sized_for_the_rows_there_are():
    """One ungrouped query: a part is one row of each head, of chunks of at
    least 64 keys."""
    f, _ = sp.spconv_attention_workspace(_attention(total_q=1, total_k=64000, batch=1, heads=4, kv_heads=4))
    assert 0 < f <= (1000 + 3) * 4 * (32 + 1) * 4


def test_size_refusals():
    assert _status(sp.spconv_attention_workspace, _attention(heads=5)) == "SPCONV_ERR_INVALID_ARG"
    assert _status(sp.spconv_attention_workspace, _attention(head_dim=4)) == "SPCONV_ERR_UNSUPPORTED"
    assert sp.STATUS[sp.lib().spconv_attention_workspace(None, None, None)] == "SPCONV_ERR_INVALID_ARG"
    assert _status(sp.spconv_norm_rotary_workspace, 12) == "SPCONV_ERR_UNSUPPORTED"
    assert sp.STATUS[sp.lib().spconv_norm_rotary_workspace(32, None)] == "SPCONV_ERR_INVALID_ARG"


@pytest.mark.parametrize("place,short", [(0, 0), (20 * FAKE, 1), (20 * FAKE + 8, 0), (FAKE, 0), (4 * FAKE - 64, 0), (5 * FAKE, 0)])
def test_refused_workspaces_of_attention(place, short):
    """NULL, too small by a byte, misaligned, and over a tensor."""
    bad = "SPCONV_ERR_INVALID_ARG"
    few = _attention(total_q=8, total_k=80000, batch=8)
    few.k, few.v = 64 * FAKE, 128 * FAKE
    need = sp.spconv_attention_workspace(few)[0]
    assert _status(sp.spconv_attention_forward_noalloc, few, 4 * FAKE, 5 * FAKE, place, need - short, 0) == bad
    a = _attention()
    need = sp.spconv_attention_workspace(a)[1]
    assert _status(sp.spconv_attention_backward_noalloc, a, 4 * FAKE, 5 * FAKE, _gradients(), place, need - short, 0) == bad
    assert _status(sp.spconv_attention_backward_noalloc, a, 4 * FAKE, 5 * FAKE, _gradients(), 9 * FAKE, need, 0) == bad


@pytest.mark.parametrize("place,short", [(0, 0), (20 * FAKE, 1), (20 * FAKE + 8, 0), (FAKE, 0), (9 * FAKE, 0)])
def test_refused_workspaces_of_the_norms_gradient(place, short):
    g = sp.spconv_norm_rotary_gradients(grad_q_out=6 * FAKE, grad_k_out=7 * FAKE, grad_q_out_row_stride=128, grad_q_out_head_stride=32,
                                        grad_k_out_row_stride=64, grad_k_out_head_stride=32, grad_q=8 * FAKE, grad_k=9 * FAKE,
                                        grad_q_row_stride=128, grad_q_head_stride=32, grad_k_row_stride=64, grad_k_head_stride=32,
                                        grad_q_weight=10 * FAKE, grad_k_weight=11 * FAKE)
    need = sp.spconv_norm_rotary_workspace(32)
    assert _status(sp.spconv_norm_rotary_backward_noalloc, _norm(), g, place, need - short, 0) == "SPCONV_ERR_INVALID_ARG"
