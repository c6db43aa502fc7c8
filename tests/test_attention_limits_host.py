"""Calls that are larger than a launch can be: refused before any device work,
on the CPU."""
import pytest

import submanifold_sparse_convolution_device_amd as sp
from test_attention_abi_host import FAKE, _attention, _norm, _status

BAD = "SPCONV_ERR_INVALID_ARG"
FAR = 1 << 44  # tensors that do not meet


@pytest.mark.parametrize("sizes", [
    dict(batch=1 << 24, heads=32, kv_heads=32, total_q=10, total_k=12),  # 2^29 tiles
    dict(batch=1 << 22, heads=1, kv_heads=1, total_q=1 << 24, total_k=1 << 30),  # few queries: a workgroup each in the join
    dict(batch=1 << 16, heads=2, kv_heads=1, total_q=(1 << 30) - 1024, total_k=5),  # nearly 2^31 rows of heads
])
def test_attention_launches(sizes):
    a = _attention(q=FAR, k=2 * FAR, v=3 * FAR, q_row_stride=1024, k_row_stride=1024, v_row_stride=1024, **sizes)
    assert _status(sp.spconv_attention_forward, a, 4 * FAR, 5 * FAR, 0) == BAD
    g = sp.spconv_attention_gradients(grad_out=6 * FAR, grad_q=7 * FAR, grad_k=8 * FAR, grad_v=9 * FAR)
    for n in ("grad_out", "grad_q", "grad_k", "grad_v"):
        setattr(g, n + "_row_stride", 1024)
        setattr(g, n + "_head_stride", 32)
    if sizes["batch"] != 1 << 22:  # (the gradient has no join there)
        assert _status(sp.spconv_attention_backward, a, 4 * FAR, 5 * FAR, g, 0) == BAD


def test_norm_rotary_launches():
    a = _norm(q=FAR, k=0, q_heads=1, k_heads=0, head_dim=128, q_row_stride=128, q_head_stride=128, rows=1 << 30, dtype=0, rotary_dim=0)
    assert _status(sp.spconv_norm_rotary_forward, a, 2 * FAR, 128, 128, 0, 0, 0, 0) == BAD


def test_rotary_table_launches():
    assert _status(sp.spconv_rotary_table, FAKE, 1 << 24, 1 << 8, 1e4, 1.0, 0) == BAD
