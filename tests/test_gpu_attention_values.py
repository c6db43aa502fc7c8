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


# ------------------------------------------------------------------ scores of minus infinity


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [32, 72, 128])
@pytest.mark.parametrize("n,at", [(400, 10), (400, 300), (1100, 300)])
@pytest.mark.parametrize("how", [dict(causal=True), dict(window=(40, 0)), dict(window=(-1, 25))])
def test_one_infinite_component_of_a_key(sp, dtype, dim, n, at, how):
    """A key with one infinite component where every query is negative: its
    scores are -inf and its probabilities 0, so it changes nothing, but for
    0 x inf = NaN in that column of the gradients of the queries that see it.
    In fp32 such a score is NaN, and so are the rows that see it."""
    cu, col = ref.offsets([n]), 5
    q, k, v = _inputs(dim + n, n, n, 2, 1, dim, dtype)[0]
    grad = torch.randn(n, 2, dim, generator=torch.Generator().manual_seed(at)).to(DT[dtype])
    q[:, :, col] = -1.0
    k[at, 0, col] = 300.0 * dim ** 0.5  # a score near -300: a probability of 0 as well
    want = ref.attention(q, k, v, cu, cu, grad=grad, **how)
    k[at, 0, col] = math.inf
    dev = tuple(t.to(DEV) for t in (q, k, v))
    out, lse = sp.attention(*dev, cu.to(DEV), return_lse=True, **how)
    gq, gk, gv = sp.attention_backward(grad.to(DEV), *dev, out, lse, cu.to(DEV), **how)
    sees = ref.visible(n, n, how.get("causal", False), how.get("window", (-1, -1)))[:, at]
    if dtype == "f32":
        for x in (out, lse, gq):
            assert bool(torch.isnan(x[sees.to(DEV)]).all())
        _near("out", out[~sees.to(DEV)], want["out"][~sees], want["out_tol"][~sees])
        _near("grad_q", gq[~sees.to(DEV)], want["grad_q"][~sees], want["grad_q_tol"][~sees])
        return
    _near("out", out, want["out"], want["out_tol"])
    _near("lse", lse, want["lse"], want["lse_tol"])
    assert bool(torch.isnan(gq[sees.to(DEV)][..., col]).all())
    hit = torch.zeros(n, 2, dim, dtype=torch.bool)
    hit[sees, :, col] = True
    _near("grad_q", gq[~hit.to(DEV)], want["grad_q"][~hit], want["grad_q_tol"][~hit])
    assert bool((gk[at] == 0).all()) and bool((gv[at] == 0).all())
    rest = torch.arange(n) != at
    _near("grad_k", gk[rest.to(DEV)], want["grad_k"][rest], want["grad_k_tol"][rest])
    _near("grad_v", gv[rest.to(DEV)], want["grad_v"][rest], want["grad_v_tol"][rest])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nq,nk,some", [(300, 300, 0), (1100, 1100, 0), (1, 3000, 0), (1, 3000, 1700), (1100, 1100, 900), (3, 400, 0)])
def test_rows_whose_scores_are_all_minus_infinity(sp, dtype, nq, nk, some):
    """Keys of which all (but one, `some`) score -inf with every query: no
    probabilities, so NaN and lse -inf, or all weight on the one key.  Rows
    that see no key stay 0.  In one pass, in splits and by parts."""
    cu_q, cu_k = ref.offsets([nq, 2]), ref.offsets([nk, 0])
    q, k, v = _inputs(nq + nk, nq + 2, nk, 2, 1, 32, dtype)[0]
    q[:, :, 5] = -1.0
    k[:, 0, 5] = math.inf
    if some:
        k[some, 0, 5] = 0.5
    dev = tuple(t.to(DEV) for t in (q, k, v))
    out, lse = sp.attention(*dev, cu_q.to(DEV), cu_k.to(DEV), return_lse=True)
    assert bool((out[nq:] == 0).all()) and bool((lse[nq:] == -math.inf).all())
    if some:
        score = (q[:nq].double() * k[some, 0].double()).sum(-1) / 32 ** 0.5
        assert torch.allclose(lse[:nq].double().cpu(), score, rtol=0, atol=80 * 2.0 ** -24 * 8)
        assert bool(((out[:nq].double().cpu() - v[some].double()).abs() <= 2 * ref.U[DT[dtype]] * v[some].double().abs() + ref.tiny(DT[dtype])).all())
        return
    assert bool(torch.isnan(out[:nq]).all()) and bool((lse[:nq] == -math.inf).all())
    grads = sp.attention_backward(torch.randn(q.shape).to(DT[dtype]).to(DEV), *dev, out, lse, cu_q.to(DEV), cu_k.to(DEV))
    assert bool(torch.isnan(grads[0][:nq]).all()) and bool((grads[0][nq:] == 0).all())
    assert bool(torch.isnan(grads[1]).all()) and bool(torch.isnan(grads[2]).all())


@pytest.mark.parametrize("nq,nk", [(40, 40), (1, 3000)])
def test_scores_beyond_fp32_are_not_zeros(sp, nq, nk):
    """Finite operands whose scaled score is not an fp32 number: NaN, not the
    result of a row without keys."""
    q, k = torch.full((nq, 1, 16), 3e18, device=DEV), torch.full((nk, 1, 16), 3e18, device=DEV)
    out, lse = sp.attention(q, k, k, ref.offsets([nq]).to(DEV), ref.offsets([nk]).to(DEV), scale=4.0, return_lse=True)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


# ------------------------------------------------------------------ lse


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("longest", [256, 1500])
def test_lse_is_not_biased(sp, dtype, longest):
    """Equal scores s of n keys: lse = s + ln n.  Its roundings have either
    sign, so their mean over many (n, s) is near 0.  In units of 2^-24 lse:
    single errors of up to about 3 leave 3 / sqrt(1800) = 0.07 of the mean; the
    logarithm of a mantissa, of size 1 or less and off by up to one unit in its
    last place, leaves up to 2^-24 ln 2 of about 5, 0.14; together 0.25.  (The
    gradients take exp(s - lse): a bias there is one of every gradient.)
    longest 1500: by parts, which are joined."""
    lengths = list(range(20, 256)) if longest == 256 else list(range(300, 1500, 5))
    pairs = [(n, s) for n in lengths for s in (0.0, 0.375, 0.5, 1.0, 1.25, 2.5, 3.0, 4.0)]
    cu_k = ref.offsets([n for n, _ in pairs])
    q, k = torch.zeros(len(pairs), 1, 8), torch.zeros(int(cu_k[-1]), 1, 8)
    q[:, 0, 2], k[:, 0, 2] = torch.tensor([s for _, s in pairs]), 1.0
    q, k = q.to(DT[dtype]).to(DEV), k.to(DT[dtype]).to(DEV)
    _, lse = sp.attention(q, k, k, ref.offsets([1] * len(pairs)).to(DEV), cu_k.to(DEV), scale=1.0, return_lse=True)
    want = torch.tensor([s + math.log(n) for n, s in pairs], dtype=torch.float64)
    off = (lse.double().cpu()[:, 0] - want) / want / 2.0 ** -24
    print(f"[lse] {dtype} {longest}: mean {float(off.mean()):.3f}, largest {float(off.abs().max()):.2f}")
    assert abs(float(off.mean())) <= 0.25


# ------------------------------------------------------------------ fp32 products


def test_fp32_products_at_the_worst_mantissas(sp):
    """One key whose score is the single product a b: what the products of
    three-part operands leave out is at most 2^-24 of it.  lse = ln 2 x (scale
    log2(e) x a b): beside that, one rounding of the product's sum (two
    allowed, 2^-24 each, for the order in the matrix unit), one of the
    multiplication by the constant and one by ln 2."""
    e = 2.0 ** -24
    values = [1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -7 + 2.0 ** -8 - 2.0 ** -16 - 2.0 ** -23, 1 + 2.0 ** -8 - 2.0 ** -23, 2 - 2.0 ** -23,
              1 + 2.0 ** -15 - 2.0 ** -23, 1.0, 4 / 3, 1.9921865]
    g = torch.Generator().manual_seed(1)
    a = torch.cat([torch.tensor(values, dtype=torch.float64), 1 + torch.rand(2000, generator=g, dtype=torch.float64)]).float()
    n = len(a)
    cu = ref.offsets([1] * n)
    c = torch.tensor(1.0, dtype=torch.float32) * torch.tensor(1.4426950408889634, dtype=torch.float32)
    ln2 = torch.tensor(0.6931471805599453, dtype=torch.float32)
    for b in (a, a.flip(0)):
        q, k = torch.zeros(n, 1, 8), torch.zeros(n, 1, 8)
        q[:, 0, 3], k[:, 0, 3] = a, b
        _, lse = sp.attention(q.to(DEV), k.to(DEV), k.to(DEV), cu.to(DEV), scale=1.0, return_lse=True)
        got = lse.double().cpu()[:, 0] / (float(c) * float(ln2))
        exact = a.double() * b.double()
        off = ((got - exact).abs() / exact) / e
        assert float(off.max()) <= 5.0, f"{float(off.max()):.2f} x 2^-24 of the product"


def test_fp32_operands_over_the_whole_range(sp):
    """The largest and smallest normal values: the three parts of an operand
    hold them without overflow, seen or hidden."""
    top = torch.finfo(torch.float32).max
    cu = ref.offsets([80]).to(DEV)
    q, k, v = torch.zeros(80, 1, 16), torch.zeros(80, 1, 16), torch.ones(80, 1, 16)
    v[:, 0, 0], v[:, 0, 1], v[:, 0, 2], v[::2, 0, 3] = top, -top, 2.0 ** -120, -top
    # every row sees itself: weight 1, and the sum of the parts is the value
    out = sp.attention(q.to(DEV), k.to(DEV), v.to(DEV), cu, window=(0, 0)).cpu()
    assert torch.equal(out, v)
    # causal: the largest values of the keys after a row leave it alone (40 equal weights of 1: 48 roundings at most)
    v = torch.ones(80, 1, 16)
    v[40:] = -top
    out = sp.attention(q.to(DEV), k.to(DEV), v.to(DEV), cu, causal=True).double().cpu()
    assert bool(((out[:40] - 1).abs() <= 48 * 2.0 ** -24).all())
    # a product of the largest and a small value: equal scores of 4
    q[:, 0, 1], k[:, 0, 1] = top, 2.0 ** -126
    _, lse = sp.attention(q.to(DEV), k.to(DEV), v.to(DEV), cu, scale=1.0, return_lse=True)
    want = top * 2.0 ** -126 + math.log(80)
    assert bool(((lse.double().cpu() - want).abs() <= 100 * 2.0 ** -24 * want).all())


@pytest.mark.parametrize("value", [-1.0, -1.2345678, 0.0, 1.2345678])
@pytest.mark.parametrize("n", [50, 300])
def test_fp32_scores_of_an_infinite_key_are_nan(sp, value, n):
    """Whatever the query's mantissa and sign."""
    cu = ref.offsets([n]).to(DEV)
    q, k, v = (t.clone() for t in _inputs(n, n, n, 1, 1, 32, "f32")[1])
    q[:, :, 4] = value
    k[n // 2, 0, 4] = math.inf
    out, lse = sp.attention(q, k, v, cu, causal=True, return_lse=True)
    assert bool(torch.isnan(out[n // 2:]).all()) and bool(torch.isnan(lse[n // 2:]).all())
    assert bool(torch.isfinite(out[:n // 2]).all())


# ------------------------------------------------------------------ time


@pytest.mark.parametrize("dtype,causal", [("f32", False), ("f32", True), ("bf16", True)])
def test_one_bad_value_costs_little(sp, dtype, causal):
    """A value that is not finite is looked for in its own tile only: less than
    three times a clean call, where going over every key again took 8 to 11
    times one (4 in bf16)."""
    n = 8000
    q, k, v = _inputs(7, n, n, 2, 2, 64, dtype)[1]
    cu = ref.offsets([n]).to(DEV)
    bad = v.clone()
    bad[n // 2, 0, 3] = math.nan

    def fastest(x):
        times = []
        for _ in range(8):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            sp.attention(q, k, x, cu, causal=causal)
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        return min(times)

    assert fastest(bad) < 3 * fastest(v)
