"""Attention over packed sequences on the GPU against the 64-bit reference
(bounds derived in attention_reference.py), at the lengths, masks, head
layouts and strides where it can go wrong."""
import math

import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EDGES = [0, 1, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 2]
NO_WINDOW = (-1, -1)


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


def _inputs(seed, nq, nk, heads, kv_heads, dim, dtype, fused=False):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    if fused:
        x = torch.randn(nq, heads + 2 * kv_heads, dim, generator=g).to(dt)
        q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
        xd = x.to(DEV)
        dev = (xd[:, :heads], xd[:, heads:heads + kv_heads], xd[:, heads + kv_heads:])
    else:
        q = torch.randn(nq, heads, dim, generator=g).to(dt)
        k = torch.randn(nk, kv_heads, dim, generator=g).to(dt)
        v = torch.randn(nk, kv_heads, dim, generator=g).to(dt)
        dev = tuple(t.to(DEV) for t in (q, k, v))
    return (q, k, v), dev, torch.randn(nq, heads, dim, generator=g).to(dt)


def _near(name, got, want, tol):
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinities differ"
    diff = torch.where(inf, 0.0, got - torch.where(inf, 0.0, want)).abs()
    assert bool((diff <= tol).all()), (f"{name}: |err| {float(diff.max()):.3e}, at most {float((diff / tol.clamp(min=1e-300)).max()):.2f} "
                                       f"times its bound")


def _check(sp, host, dev, grad, cu_q, cu_k, backward=True, **how):
    print(f"[attention] {host[0].dtype} q{tuple(host[0].shape)} k{tuple(host[1].shape)} {len(cu_q) - 1} sequences {how}", flush=True)
    want = ref.attention(*host, cu_q, cu_k, grad=grad if backward else None, **how)
    cq, ck = cu_q.to(DEV), cu_k.to(DEV)
    out, lse = sp.attention(*dev, cq, ck, return_lse=True, **how)
    _near("out", out, want["out"], want["out_tol"])
    _near("lse", lse, want["lse"], want["lse_tol"])
    if backward:
        got = sp.attention_backward(grad.to(DEV), *dev, out, lse, cq, ck, **how)
        for n, x in zip(("grad_q", "grad_k", "grad_v"), got):
            _near(n, x, want[n], want[n + "_tol"])
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 16, 32, 40, 64, 72, 96, 120, 128])
def test_lengths_around_the_tiles(sp, dtype, dim):
    cu = ref.offsets(EDGES)
    n = int(cu[-1])
    host, dev, grad = _inputs(dim, n, n, 2, 2, dim, dtype)
    _check(sp, host, dev, grad, cu, cu)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 32), (6, 2, 64), (8, 8, 16), (5, 1, 128), (7, 7, 24)])
@pytest.mark.parametrize("how", [dict(causal=True), dict(window=(20, 7)), dict(window=(0, 0)), dict(causal=True, window=(50, -1)),
                                 dict(window=(-1, 40)), dict(window=(200, -1))])
def test_masks_and_grouped_heads(sp, dtype, heads, kv_heads, dim, how):
    cu = ref.offsets([1, 300, 0, 65, 129])
    n = int(cu[-1])
    host, dev, grad = _inputs(heads * dim, n, n, heads, kv_heads, dim, dtype, fused=True)
    _check(sp, host, dev, grad, cu, cu, **how)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("how", [dict(), dict(causal=True), dict(window=(3, 3)), dict(causal=True, window=(0, -1))])
def test_other_keys_and_rows_that_see_none(sp, dtype, how):
    """Queries without keys, keys without queries, and more queries than keys
    (under a causal mask the first ones see nothing)."""
    cu_q = ref.offsets([5, 0, 70, 33, 1, 100])
    cu_k = ref.offsets([0, 9, 40, 150, 1, 3])
    host, dev, grad = _inputs(11, int(cu_q[-1]), int(cu_k[-1]), 4, 2, 40, dtype)
    out, lse = _check(sp, host, dev, grad, cu_q, cu_k, **how)
    assert bool((out[:5] == 0).all()) and bool((lse[:5] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,queries", [(16, 2, 128, 1), (4, 4, 32, 1), (3, 1, 64, 2), (8, 1, 96, 5)])
def test_single_queries_over_long_keys(sp, dtype, heads, kv_heads, dim, queries):
    """A new row, or a few, of each sequence against the rows before it."""
    lengths = [1, 5000, 0, 700, 33, 2049]
    cu_q, cu_k = ref.offsets([queries] * len(lengths)), ref.offsets(lengths)
    host, dev, grad = _inputs(heads, int(cu_q[-1]), int(cu_k[-1]), heads, kv_heads, dim, dtype)
    _check(sp, host, dev, grad, cu_q, cu_k, causal=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_of_no_sequence(sp, dtype):
    """Rows before the first offset and after the last one."""
    cu_q, cu_k = ref.offsets([30, 65], 7), ref.offsets([50, 40], 3)
    host, dev, grad = _inputs(3, int(cu_q[-1]) + 70, int(cu_k[-1]) + 130, 2, 1, 32, dtype)
    out, lse = _check(sp, host, dev, grad, cu_q, cu_k)
    assert bool((out[:7] == 0).all()) and bool((lse[-70:] == -math.inf).all())


@pytest.mark.parametrize("batch", [0, 1, 63, 64, 200, 5000])
def test_many_sequences(sp, batch):
    g = torch.Generator().manual_seed(batch)
    lengths = torch.randint(0, 6, (batch,), generator=g).tolist()
    cu = ref.offsets(lengths)
    n = int(cu[-1]) + 2
    host, dev, grad = _inputs(batch, n, n, 2, 2, 16, "bf16")
    _check(sp, host, dev, grad, cu, cu, causal=True)


def test_no_rows(sp):
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    q = torch.empty(0, 4, 32, dtype=torch.bfloat16, device=DEV)
    k = torch.randn(6, 2, 32, device=DEV).bfloat16()
    out, lse = sp.attention(q, k, k, cu, cu, return_lse=True)
    assert out.shape == (0, 4, 32) and lse.shape == (0, 4)
    gq, gk, gv = sp.attention_backward(q, q, k, k, out, lse, cu, cu)
    assert gq.shape == q.shape and bool((gk == 0).all()) and bool((gv == 0).all())
    q = torch.randn(5, 4, 32, device=DEV).bfloat16()
    e = torch.empty(0, 2, 32, dtype=torch.bfloat16, device=DEV)
    out, lse = sp.attention(q, e, e, cu, cu, return_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    gq, gk, gv = sp.attention_backward(q, q, e, e, out, lse, cu, cu)
    assert bool((gq == 0).all()) and gk.shape == e.shape


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strides_and_repeated_heads(sp, dtype):
    """Heads before rows, padded rows, a key head repeated by stride 0, and
    gradients into the slices of one buffer."""
    cu = ref.offsets([40, 100, 3])
    n = int(cu[-1])
    dt = DT[dtype]
    g = torch.Generator().manual_seed(5)
    q = torch.randn(3, n, 48, generator=g).to(dt)  # [heads, rows, dim]
    k = torch.randn(n, 1, 64, generator=g).to(dt)  # 16 elements after each row
    v = torch.randn(n, 3, 48, generator=g).to(dt)
    grad = torch.randn(n, 3, 48, generator=g).to(dt)
    qd, kd, vd = q.to(DEV).transpose(0, 1), k.to(DEV)[..., :48].expand(n, 3, 48), v.to(DEV)
    host = (q.transpose(0, 1), k[..., :48].expand(n, 3, 48), v)
    assert kd.stride(1) == 0
    want = ref.attention(*host, cu, cu, causal=True, grad=grad)
    c = cu.to(DEV)
    out, lse = sp.attention(qd, kd, vd, c, causal=True, return_lse=True)
    _near("out", out, want["out"], want["out_tol"])
    into = torch.full((n, 9, 48), 7.0, dtype=dt, device=DEV)
    sp.attention_backward(grad.to(DEV), qd, kd, vd, out, lse, c, causal=True, grads=(into[:, :3], into[:, 3:6], into[:, 6:]))
    for i, name in enumerate(("grad_q", "grad_k", "grad_v")):
        _near(name, into[:, 3 * i:3 * i + 3], want[name], want[name + "_tol"])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("magnitude", [1e-4, 1.0, 200.0])
def test_gradients_of_any_magnitude(sp, dtype, magnitude):
    """Gradients whose score gradients leave fp16's normal range at both ends."""
    cu = ref.offsets([900, 17])
    n = int(cu[-1])
    host, dev, grad = _inputs(9, n, n, 2, 1, 32, dtype)
    _check(sp, host, dev, (grad.float() * magnitude).to(DT[dtype]), cu, cu)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_large_scores(sp, dtype):
    """Scores of hundreds, growing along the keys, so that the running maximum
    moves in every tile; a scale of the caller's."""
    cu = ref.offsets([500])
    host, dev, grad = _inputs(4, 500, 500, 1, 1, 32, dtype)
    ramp = torch.linspace(0.1, 10, 500)[:, None, None]
    k = (host[1].float() * ramp).to(DT[dtype])
    host = (host[0], k, host[2])
    _check(sp, host, (dev[0], k.to(DEV), dev[2]), grad, cu, cu, scale=0.5)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_other_sequences_values_do_not_leak(sp, dtype):
    """NaN and infinities in one sequence stay there, forward and backward."""
    cu = ref.offsets([33, 40, 21])
    host, dev, grad = _inputs(6, 94, 94, 2, 2, 32, dtype)
    for t in dev:
        t[33:73] = float("nan")
        t[40:50] = float("inf")
    grad = grad.to(DEV)
    grad[33:73] = float("nan")
    c = cu.to(DEV)
    out, lse = sp.attention(*dev, c, causal=True, return_lse=True)
    got = sp.attention_backward(grad, *dev, out, lse, c, causal=True)
    want = ref.attention(*(t[:33] for t in host), cu[:2], cu[:2], causal=True, grad=grad[:33].cpu())
    for n, x in zip(("out", "grad_q", "grad_k", "grad_v"), (out, *got)):
        assert bool(torch.isfinite(x[:33]).all()) and bool(torch.isfinite(x[73:]).all()), n
        _near(n, x[:33], want[n], want[n + "_tol"])
    assert bool(torch.isnan(out[33:73]).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [3, 40, 150])
def test_one_row_repeated(sp, dtype, n):
    """Keys and values that repeat one row (row stride 0), an infinity in it:
    every query gets that row, whatever tiles the sequence ends in."""
    cu = ref.offsets([n]).to(DEV)
    host, dev, grad = _inputs(n, n, 1, 2, 2, 48, dtype)
    k = dev[1].expand(n, 2, 48)
    v = dev[2].clone()
    v[0, 1, 5] = math.inf
    v = v.expand(n, 2, 48)
    assert k.stride(0) == 0 and v.stride(0) == 0
    out, lse = sp.attention(dev[0], k, v, cu, return_lse=True)
    # equal scores: weights 1 / n each, in one order of sums (and the rounding to dtype, at most |v| eps)
    eps = torch.finfo(DT[dtype]).eps
    bound = (4 * eps + 2.0 ** -20) * host[2].double().abs().expand(n, 2, 48) + 1e-30
    want = v.double().cpu()
    _near("out", out, want, torch.where(torch.isinf(want), 1.0, bound))
    # a key with an infinity: no query's gradient is finite where its scores are not, and none hangs on it elsewhere
    bad = dev[1].clone()
    bad[0, 0, 7] = math.inf
    o, l = sp.attention(dev[0], bad.expand(n, 2, 48), dev[2].expand(n, 2, 48), cu, return_lse=True)
    gq, _, _ = sp.attention_backward(grad.to(DEV), dev[0], bad.expand(n, 2, 48), dev[2].expand(n, 2, 48), o, l, cu)
    assert bool(torch.isfinite(gq[:, 1]).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [32, 72, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [40, 200])
def test_hidden_values_do_not_leak(sp, dtype, dim, value, n):
    """A value that is not finite in one row reaches the queries that see the
    row, in its own column, and no other ones: forward (v), and of the
    gradients those of rows that neither see it nor are seen by it."""
    cu = ref.offsets([n])
    host, dev, grad = _inputs(dim, n, n, 2, 1, dim, dtype)
    at, c = n - 7, cu.to(DEV)
    clean = ref.attention(*host, cu, cu, causal=True, window=(12, 0), grad=grad)
    how = dict(causal=True, window=(12, 0))
    v = dev[2].clone()
    v[at, 0, 5] = value
    out = sp.attention(dev[0], dev[1], v, c, **how)
    sees = torch.zeros(n, dtype=torch.bool)
    sees[at:min(n, at + 13)] = True
    _near("out", out[~sees.to(DEV)], clean["out"][~sees], clean["out_tol"][~sees])
    got = out[sees.to(DEV)].double().cpu()
    assert bool(torch.isnan(got[:, :, 5]).all() if math.isnan(value) else (got[:, :, 5] == value).all())
    others = [i for i in range(dim) if i != 5]
    assert bool(torch.isfinite(got[:, :, others]).all())
    # gradients: a key, and a query's output gradient
    out, lse = sp.attention(*dev, c, return_lse=True, **how)
    k = dev[1].clone()
    k[at] = value
    bad_out, bad_lse = sp.attention(dev[0], k, dev[2], c, return_lse=True, **how)
    gq, gk, gv = sp.attention_backward(grad.to(DEV), dev[0], k, dev[2], bad_out, bad_lse, c, **how)
    apart = torch.arange(n) < at - 12  # keys that no query in sight of the bad one sees
    _near("grad_q", gq[:at], clean["grad_q"][:at], clean["grad_q_tol"][:at])
    _near("grad_k", gk[apart.to(DEV)], clean["grad_k"][apart], clean["grad_k_tol"][apart])
    _near("grad_v", gv[apart.to(DEV)], clean["grad_v"][apart], clean["grad_v_tol"][apart])
    g = grad.to(DEV).clone()
    g[at, 1, 3] = value
    gq, gk, gv = sp.attention_backward(g, *dev, out, lse, c, **how)
    seen_by = torch.zeros(n, dtype=torch.bool)
    seen_by[at - 12:at + 1] = True
    rest = torch.arange(n) != at
    _near("grad_q", gq[rest.to(DEV)], clean["grad_q"][rest], clean["grad_q_tol"][rest])
    _near("grad_k", gk[~seen_by.to(DEV)], clean["grad_k"][~seen_by], clean["grad_k_tol"][~seen_by])
    _near("grad_v", gv[~seen_by.to(DEV)], clean["grad_v"][~seen_by], clean["grad_v_tol"][~seen_by])
    assert not bool(torch.isfinite(gv[seen_by.to(DEV), 0, 3]).any())
    assert not bool(torch.isfinite(gk[seen_by.to(DEV)]).any())


def test_tiles_in_order_of_work(sp):
    """Lengths and sizes for which the tiles are sorted by work first."""
    lengths = [2400, 1, 0, 130]
    cu = ref.offsets(lengths)
    n = int(cu[-1])
    host, dev, grad = _inputs(13, n, n, 8, 8, 64, "f32")
    _check(sp, host, dev, grad, cu, cu)


def test_offsets_that_break_the_rules_stay_inside(sp):
    """Decreasing, negative and too large offsets: no access outside the
    tensors (the call returns; its rows mean nothing)."""
    q = torch.randn(100, 2, 32, device=DEV).bfloat16()
    for bad in ([0, 50, 20, 100], [-7, 10, 5000, 100], [90, 10, 0, 3], [2 ** 31 - 1, -2 ** 31, 0, 100]):
        c = torch.tensor(bad, dtype=torch.int32, device=DEV)
        out, lse = sp.attention(q, q, q, c, return_lse=True)
        sp.attention_backward(q, q, q, q, torch.zeros_like(out), torch.zeros_like(lse), c)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time_and_on_another_stream(sp, dtype):
    cu_q, cu_k = ref.offsets([1, 3, 1]), ref.offsets([4000, 100, 900])
    host, dev, grad = _inputs(8, 5, 5000, 8, 2, 64, dtype)
    cq, ck, g = cu_q.to(DEV), cu_k.to(DEV), grad.to(DEV)

    def step():
        out, lse = sp.attention(*dev, cq, ck, causal=True, return_lse=True)
        return (out, lse, *sp.attention_backward(g, *dev, out, lse, cq, ck, causal=True))

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = step()
    third = step()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_gradients_against_differences(sp):
    """fp32 gradients along random directions against central differences of
    the 64-bit forward."""
    cu = ref.offsets([9, 1, 20])
    host, dev, grad = _inputs(21, 30, 30, 4, 2, 16, "f32")
    c = cu.to(DEV)
    out, lse = sp.attention(*dev, c, causal=True, return_lse=True)
    got = sp.attention_backward(grad.to(DEV), *dev, out, lse, c, causal=True)
    tol = ref.attention(*host, cu, cu, causal=True, grad=grad)
    g = torch.Generator().manual_seed(3)
    h = 1e-5
    for at, name in enumerate(("grad_q", "grad_k", "grad_v")):
        u = torch.randn(host[at].shape, generator=g, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            x = [t.double() for t in host]
            x[at] = x[at] + sign * h * u
            # the bounds of a 64-bit "dtype" are not used here
            o = _forward64(x, cu)
            ends.append(float((o * grad.double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        mine = float((got[at].double().cpu() * u).sum())
        # the gradient's own bound along u, and the quotient's h^2 and rounding terms
        assert abs(mine - slope) <= float((tol[name + "_tol"] * u.abs()).sum()) + 1e-6 * (1 + abs(slope)), name


def _forward64(x, cu):
    q, k, v = x
    out = torch.zeros_like(q)
    for b in range(len(cu) - 1):
        s = slice(int(cu[b]), int(cu[b + 1]))
        n = s.stop - s.start
        for h in range(q.shape[1]):
            a = q[s, h] @ k[s, h // 2].T / 4.0
            a = a.masked_fill(torch.ones(n, n).triu(1).bool(), -math.inf)
            out[s, h] = torch.softmax(a, -1) @ v[s, h // 2]
    return out


def test_captured_in_a_graph(sp):
    """The calls replay from a captured graph, with other values each time."""
    cu = ref.offsets([100, 30]).to(DEV)
    _, dev, grad = _inputs(2, 130, 130, 4, 2, 32, "bf16")
    q, k, v = dev
    grad = grad.to(DEV)

    def step():
        out, lse = sp.attention(q, k, v, cu, causal=True, return_lse=True)
        return (out, *sp.attention_backward(grad, q, k, v, out, lse, cu, causal=True))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # the stream's workspace grows before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    for i in range(4):
        q.copy_(torch.randn(q.shape, device=DEV))
        v.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b), i


def test_refusals(sp):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, k = torch.zeros(10, 4, 32, **bf), torch.zeros(10, 2, 32, **bf)
    cu = torch.tensor([0, 10], dtype=torch.int32, device=DEV)

    def status(*a, **kw):
        with pytest.raises(sp.SpconvError) as e:
            sp.attention(*a, **kw)
        return e.value.name

    assert status(q.double(), k.double(), k.double(), cu) == "SPCONV_ERR_UNSUPPORTED"
    assert status(torch.zeros(10, 4, 136, **bf), torch.zeros(10, 2, 136, **bf), torch.zeros(10, 2, 136, **bf), cu) == "SPCONV_ERR_UNSUPPORTED"
    assert status(torch.zeros(10, 4, 12, **bf), torch.zeros(10, 2, 12, **bf), torch.zeros(10, 2, 12, **bf), cu) == "SPCONV_ERR_UNSUPPORTED"
    three = torch.zeros(10, 3, 32, **bf)
    assert status(q, three, three, cu) == "SPCONV_ERR_INVALID_ARG"
    for bad in ((q.float(), k, k, cu), (q, k, k[:9], cu), (q, k, torch.zeros(10, 2, 40, **bf), cu), (q.cpu(), k, k, cu),
                (q, k, k, cu.long()), (q, k, k, cu.cpu()), (q, k, k, cu, torch.cat([cu, cu])), (q[0], k, k, cu),
                (torch.zeros(10, 4, 64, **bf)[..., ::2], k, k, cu), (torch.zeros(10, 4, 36, **bf)[..., 4:], k, k, cu),
                (torch.zeros(10 * 132, **bf)[:1320].view(10, 132)[:, :128].view(10, 4, 32), k, k, cu)):
        assert status(*bad) == "SPCONV_ERR_INVALID_ARG"
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert status(q, k, k, cu, scale=scale) == "SPCONV_ERR_INVALID_ARG"
    assert status(q, k, k, cu, out=q) == "SPCONV_ERR_INVALID_ARG"
    out, lse = sp.attention(q, k, k, cu, return_lse=True)

    def status_b(*a, **kw):
        with pytest.raises(sp.SpconvError) as e:
            sp.attention_backward(*a, **kw)
        return e.value.name

    good = (q, q, k, k, out, lse, cu)
    assert status_b(q[:9], *good[1:]) == "SPCONV_ERR_INVALID_ARG"
    assert status_b(*good[:5], lse.double(), cu) == "SPCONV_ERR_INVALID_ARG"
    assert status_b(*good[:4], out.transpose(0, 1), lse, cu) == "SPCONV_ERR_INVALID_ARG"
    g = [torch.empty_like(t) for t in (q, k, k)]
    assert status_b(*good, grads=(q, g[1], g[2])) == "SPCONV_ERR_INVALID_ARG"
    assert status_b(*good, grads=(g[0], g[1], g[1])) == "SPCONV_ERR_INVALID_ARG"
    assert status_b(*good, grads=(g[0], g[1][:, :1].expand(10, 2, 32), g[2])) == "SPCONV_ERR_INVALID_ARG"
    one = torch.zeros(10, 7, 32, **bf)
    assert status_b(*good, grads=(one[:, :4], one[:, 3:5], one[:, 5:])) == "SPCONV_ERR_INVALID_ARG"
