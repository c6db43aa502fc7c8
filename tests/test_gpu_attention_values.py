"""Attention over values that are not finite, and at the ends of a type's
range: what the formulas give in 64 bits, on every path that a call can take."""
import math

import pytest
import torch

import attention_reference as ref
from test_gpu_attention import DEV, DT, _inputs, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


# ------------------------------------------------------------------ few queries over long keys


# keys of each sequence: one part (chunks are of 64 keys here), several, and more parts than one round of the join takes
LONG = [60, 5000, 700, 2049, 0]


def _check_rows(out, lse, want, bad):
    """Rows `bad` [rows, heads] are NaN in out and lse; the others are near."""
    bad = bad.to(out.device)
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all()), "a row that sees a NaN is not NaN"
    good = ~bad
    keep = good.cpu()
    _near("out", out[good], want["out"][keep], want["out_tol"][keep])
    _near("lse", lse[good], want["lse"][keep], want["lse_tol"][keep])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(16, 2, 128), (4, 4, 16), (4, 1, 64)])
def test_nan_query_over_long_keys(sp, dtype, heads, kv_heads, dim):
    """A NaN in one head of one query: NaN for that row and head alone, also
    where the sequence has a single part."""
    cu_q, cu_k = ref.offsets([1] * len(LONG)), ref.offsets(LONG)
    host, dev, _ = _inputs(dim, len(LONG), sum(LONG), heads, kv_heads, dim, dtype)
    want = ref.attention(*host, cu_q, cu_k, causal=True)
    q = dev[0].clone()
    bad = torch.zeros(len(LONG), heads, dtype=torch.bool)
    for row, head in ((0, heads - 1), (1, 0), (2, 1), (3, 0)):
        q[row, head, 3] = math.nan
        bad[row, head] = True
    out, lse = sp.attention(q, *dev[1:], cu_q.to(DEV), cu_k.to(DEV), causal=True, return_lse=True)
    _check_rows(out, lse, want, bad)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(16, 2, 128), (4, 4, 16)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("place", [0, 59, 350, 4999])
def test_bad_key_among_long_keys(sp, dtype, heads, kv_heads, dim, value, place):
    """A key whose scores are NaN, in any part: NaN for the heads that share it,
    in the sequences whose query sees it."""
    cu_q, cu_k = ref.offsets([1] * len(LONG)), ref.offsets(LONG)
    host, dev, _ = _inputs(dim + place, len(LONG), sum(LONG), heads, kv_heads, dim, dtype)
    want = ref.attention(*host, cu_q, cu_k, causal=True)
    k = dev[1].clone()
    bad = torch.zeros(len(LONG), heads, dtype=torch.bool)
    group = heads // kv_heads
    for b, n in enumerate(LONG):
        if place < n:
            k[int(cu_k[b]) + place, 0] = value  # mixed signs against any query: NaN scores
            bad[b, :group] = True
    out, lse = sp.attention(dev[0], k, dev[2], cu_q.to(DEV), cu_k.to(DEV), causal=True, return_lse=True)
    _check_rows(out, lse, want, bad)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("queries,window", [(1, (200, 0)), (1, (0, 0)), (3, (63, 0)), (5, (700, 0)), (2, (100, 30))])
def test_few_queries_with_a_band(sp, dtype, queries, window):
    """A band ends inside a part, leaves whole parts out, and hides what is not
    finite in them."""
    cu_q, cu_k = ref.offsets([queries] * len(LONG)), ref.offsets(LONG)
    host, dev, _ = _inputs(queries, queries * len(LONG), sum(LONG), 4, 2, 40, dtype)
    want = ref.attention(*host, cu_q, cu_k, window=window)
    k, v = dev[1].clone(), dev[2].clone()
    for b, n in enumerate(LONG):
        hidden = n - queries - window[0]  # the keys below the first query's band
        if hidden > 0:
            at = int(cu_k[b])
            k[at:at + hidden:7] = math.nan
            v[at:at + hidden:5] = math.inf
            v[at + hidden - 1] = math.nan
    out, lse = sp.attention(dev[0], k, v, cu_q.to(DEV), cu_k.to(DEV), window=window, return_lse=True)
    _check_rows(out, lse, want, torch.zeros(queries * len(LONG), 4, dtype=torch.bool))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_few_queries_over_strided_keys(sp, dtype):
    """Heads before rows, padded rows and one value head for all, by parts."""
    cu_q, cu_k = ref.offsets([1] * len(LONG)), ref.offsets(LONG)
    n, dt = sum(LONG), DT[dtype]
    g = torch.Generator().manual_seed(12)
    q = torch.randn(len(LONG), 6, 72, generator=g).to(dt)
    k = torch.randn(3, n, 48, generator=g).to(dt)
    v = torch.randn(n, 1, 64, generator=g).to(dt)
    host = (q[..., 8:56], k.transpose(0, 1), v[..., :48].expand(n, 3, 48))
    want = ref.attention(*host, cu_q, cu_k, causal=True)
    out, lse = sp.attention(q.to(DEV)[..., 8:56], k.to(DEV).transpose(0, 1), v.to(DEV)[..., :48].expand(n, 3, 48), cu_q.to(DEV),
                            cu_k.to(DEV), causal=True, return_lse=True)
    _check_rows(out, lse, want, torch.zeros(len(LONG), 6, dtype=torch.bool))


# ------------------------------------------------------------------ gradients of keys


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [32, 72, 128])
@pytest.mark.parametrize("nq,nk,window", [(10, 64, (5, -1)), (45, 300, (70, 0)), (300, 430, (20, -1)), (3, 40, (0, 0))])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_unseen_keys_have_zero_gradients(sp, dtype, dim, nq, nk, window, value):
    """Keys and values that are not finite and that no query sees: gradients of
    exactly 0, beside tiles of rows that end past the last query."""
    cu_q, cu_k = ref.offsets([nq, 1]), ref.offsets([nk, 30])
    host, dev, grad = _inputs(dim + nk, nq + 1, nk + 30, 2, 1, dim, dtype)
    want = ref.attention(*host, cu_q, cu_k, grad=grad, window=window)
    unseen = nk - nq - window[0]  # the first keys
    assert unseen > 0
    k, v = dev[1].clone(), dev[2].clone()
    k[:unseen:3] = value
    v[1:unseen:3] = value
    k[unseen - 1], v[unseen - 1] = value, value
    cq, ck = cu_q.to(DEV), cu_k.to(DEV)
    out, lse = sp.attention(dev[0], k, v, cq, ck, window=window, return_lse=True)
    _near("out", out, want["out"], want["out_tol"])
    got = sp.attention_backward(grad.to(DEV), dev[0], k, v, out, lse, cq, ck, window=window)
    for n, x in zip(("grad_q", "grad_k", "grad_v"), got):
        _near(n, x, want[n], want[n + "_tol"])
    assert bool((got[1][:unseen] == 0).all()) and bool((got[2][:unseen] == 0).all())
