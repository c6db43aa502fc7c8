"""Attention whose tiles run in order of falling work, against the 64-bit
reference (computed on the GPU): the order has to hold every tile once, for
grouped heads, under masks and in every type."""
import pytest
import torch

import attention_reference as ref
from test_gpu_attention import DEV, DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


def _near(name, got, want, tol):
    off = (got.double() - want).abs()
    # a tile that no workgroup took leaves NaN, which is not <= either
    assert bool((off <= tol).all()), f"{name}: |err| {float(off.max()):.3e}, {float((off / tol.clamp(min=1e-300)).max()):.2f} times its bound"


# Sizes at which both the forward (unsplit, between 512 and 2560 workgroups)
# and the gradients are sorted: the work is above the rule's thresholds.
@pytest.mark.parametrize("dtype,heads,kv_heads,dim,lengths_q,lengths_k,how", [
    ("f16", 8, 2, 64, [4100, 1, 0, 4900, 4400, 4300], None, dict(causal=True)),
    ("bf16", 8, 4, 64, [5000, 4600, 130, 5100], None, dict(window=(1500, 300))),
    ("bf16", 6, 6, 72, [5600, 33, 5600], [5200, 0, 5400], dict()),
    ("f32", 16, 4, 32, [1500, 1700, 31, 1601], [1500, 1900, 1, 1500], dict(causal=True)),
    ("f32", 12, 3, 40, [2100, 1900, 2000], None, dict(causal=True, window=(900, -1))),
])
def test_sorted_tiles(sp, dtype, heads, kv_heads, dim, lengths_q, lengths_k, how):
    lengths_k = lengths_q if lengths_k is None else lengths_k
    cu_q, cu_k = ref.offsets(lengths_q), ref.offsets(lengths_k)
    g = torch.Generator().manual_seed(dim)
    q = torch.randn(sum(lengths_q), heads, dim, generator=g).to(DT[dtype]).to(DEV)
    k, v = (torch.randn(sum(lengths_k), kv_heads, dim, generator=g).to(DT[dtype]).to(DEV) for _ in range(2))
    grad = torch.randn(sum(lengths_q), heads, dim, generator=g).to(DT[dtype]).to(DEV)
    cq, ck = cu_q.to(DEV), cu_k.to(DEV)
    sp._bind()
    packed = sp._attention_args(q, k, v, cq, ck, how.get("causal", False), how.get("window", (-1, -1)), None)
    # unsplit: the forward's workspace holds nothing but the order of the slots
    assert 0 < sp._attention_workspace(packed)[0] <= 4 * 2560
    out = torch.full_like(q, float("nan"))
    out, lse = sp.attention(q, k, v, cq, ck, out=out, return_lse=True, **how)
    grads = tuple(torch.full_like(x, float("nan")) for x in (q, k, v))
    sp.attention_backward(grad, q, k, v, out, lse, cq, ck, grads=grads, **how)
    with torch.device(DEV):
        want = ref.attention(q, k, v, cu_q, cu_k, grad=grad, **how)
    _near("out", out, want["out"], want["out_tol"])
    seen = torch.isfinite(want["lse"])
    assert torch.equal(lse[~seen].double(), want["lse"][~seen])
    _near("lse", lse[seen], want["lse"][seen], want["lse_tol"][seen])
    for n, x in zip(("grad_q", "grad_k", "grad_v"), grads):
        _near(n, x, want[n], want[n + "_tol"])
