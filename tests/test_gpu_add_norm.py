"""The residual's addition with the row norm, and its gradient, against the
formulas in 64 bits.

Bounds: the sum of squares of c values in fp32 is off by at most (c + 1) units
of 2^-24 relatively, so 1 / sqrt by half of that and a few units; the products
by a unit each.  The gradient's mean is off by (c + 4) units of the mean of
|t h|, and weight gradients by (rows + c / 2 + 8) units of the sum of sizes.
"""
import pytest
import torch

import submanifold_sparse_convolution_device_amd as sp
from linear_reference import DTYPES, UNIT, close, rounding, smallest

pytestmark = pytest.mark.gpu

CHANNELS = [8, 16, 40, 64, 96, 128, 136, 256, 264, 512, 520, 1024, 2048, 2056, 4096, 8192]
EPS = 1e-5


def _draw(dtype, *shape, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).cuda()


def _check(x, residual, w, out=None):
    c, dt = x.shape[1], x.dtype
    want = x if residual is None else (x.double() + residual.double()).to(dt)
    h, y = sp.add_norm(x, residual, w, eps=EPS, out=out)
    # (fp32 rounds the sum once; sums of 16-bit values near a tie are exact in fp32)
    assert torch.equal(h, want)
    ref = want.double()
    ref = ref / torch.sqrt((ref * ref).mean(-1, keepdim=True) + EPS) * w.double()
    close(y, ref, ref.abs() * (rounding(dt) * (1 + UNIT) + (c / 2 + 8) * UNIT) + smallest(dt), "y")
    return h, y


def _check_backward(gh, gy, h, w, **rest):
    c, dt, rows = h.shape[1], h.dtype, h.shape[0]
    gh64 = None if gh is None else gh.double()
    gy64 = gy.double()
    grad, gw = sp.add_norm_backward(gh, gy, h, w, eps=EPS, **rest)
    x, t = h.double(), gy64 * w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    m = (t * x).mean(-1, keepdim=True)
    ref = r * (t - x * r * r * m)
    size = r * (t.abs() + x.abs() * r * r * (t * x).abs().mean(-1, keepdim=True))
    if gh is not None:
        ref, size = ref + gh64, size + gh64.abs()
    bound = (2 * c + 16) * UNIT * size
    close(grad, ref, bound + rounding(dt) * (ref.abs() + bound) + smallest(dt), "grad")
    terms = gy64 * x * r
    close(gw, terms.sum(0), (rows + c / 2 + 8) * UNIT * terms.abs().sum(0), "grad_weight")
    return grad, gw


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", CHANNELS + [16384])
@pytest.mark.parametrize("rows", [1, 37])
def test_add_norm(dtype, channels, rows):
    dt = DTYPES[dtype]
    if channels * dt.itemsize > 32768:
        with pytest.raises(sp.SpconvError, match="UNSUPPORTED"):
            sp.add_norm(_draw(dt, rows, channels, seed=1), None, _draw(dt, channels, seed=2))
        return
    x, res = _draw(dt, rows, channels, seed=1), _draw(dt, rows, channels, seed=2, scale=2.0)
    w = _draw(dt, channels, seed=3, scale=0.3, shift=1.0)
    h, _ = _check(x, res, w)
    assert _check(x, None, w)[0] is x
    gh, gy = _draw(dt, rows, channels, seed=4), _draw(dt, rows, channels, seed=5)
    _check_backward(gh, gy, h, w)
    _check_backward(None, gy, h, w)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,channels", [(20011, 96), (5003, 264), (3001, 2056)])
def test_many_rows(dtype, rows, channels):
    """More rows than the gradient's workgroups hold at once."""
    dt = DTYPES[dtype]
    x, res = _draw(dt, rows, channels, seed=1), _draw(dt, rows, channels, seed=2)
    w = _draw(dt, channels, seed=3, scale=0.3, shift=1.0)
    h, _ = _check(x, res, w)
    _check_backward(_draw(dt, rows, channels, seed=4), _draw(dt, rows, channels, seed=5), h, w)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [48, 1000, 4096])
def test_places_and_strides(dtype, channels):
    dt = DTYPES[dtype]
    rows = 30
    w = _draw(dt, channels, seed=3, shift=1.0)
    wide = [_draw(dt, rows, channels + 16, seed=s) for s in range(4)]
    x, res = wide[0][:, 8:8 + channels], wide[1][:, :channels]
    h, y = _check(x, res, w)
    a, b = x.clone(), res.clone()
    got = sp.add_norm(a, b, w, eps=EPS, out=(b, a))  # the sum in the residual's place, the norm in x's
    assert torch.equal(b, h) and torch.equal(a, y) and got[0] is b
    around = wide[0].clone()
    sp.add_norm(x, None, w, eps=EPS, out=(None, x))
    assert torch.equal(wide[0][:, :8], around[:, :8]) and torch.equal(wide[0][:, 8 + channels:], around[:, 8 + channels:])
    gh, gy = wide[2][:, :channels], wide[3][:, 8:8 + channels]
    grad, gw = _check_backward(gh, gy, h, w)
    for place in (gh, gy):
        p, q = (gh.clone(), gy.clone())
        into = p if place is gh else q
        again, gw2 = sp.add_norm_backward(p, q, h, w, eps=EPS, grad=into)
        assert again is into and torch.equal(again, grad) and torch.equal(gw, gw2)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_no_rows_and_zero_rows(dtype):
    dt = DTYPES[dtype]
    w = _draw(dt, 40, seed=1)
    empty = torch.empty(0, 40, dtype=dt, device="cuda")
    h, y = sp.add_norm(empty, empty.clone(), w)
    grad, gw = sp.add_norm_backward(None, y, h, w)
    assert grad.shape == (0, 40) and not bool(gw.any())
    zero = torch.zeros(9, 40, dtype=dt, device="cuda")
    h, y = sp.add_norm(zero, zero.clone(), w, eps=EPS)
    assert not bool(y.any())
    _check_backward(None, _draw(dt, 9, 40, seed=2), h, w)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_values_that_are_not_finite_stay_in_their_row(dtype):
    dt = DTYPES[dtype]
    x, res, w = _draw(dt, 100, 96, seed=1), _draw(dt, 100, 96, seed=2), _draw(dt, 96, seed=3)
    h0, y0 = sp.add_norm(x, res, w)
    x[7, 5], x[63, 0] = float("nan"), float("inf")
    h, y = sp.add_norm(x, res, w)
    keep = torch.ones(100, dtype=torch.bool, device="cuda")
    keep[7] = keep[63] = False
    assert torch.equal(y[keep], y0[keep]) and bool(y[7].isnan().all()) and bool(y[63, 0].isnan()) and not bool(y[63, 1:].any())
    g = _draw(dt, 100, 96, seed=4)
    a, _ = sp.add_norm_backward(None, g, h0, w)
    b, _ = sp.add_norm_backward(None, g, h, w)
    assert torch.equal(a[keep], b[keep]) and bool(b[7].isnan().all())


def test_against_differences():
    x = _draw(torch.float32, 5, 24, seed=1)
    w, seed = _draw(torch.float32, 24, seed=2, shift=1.0), _draw(torch.float32, 5, 24, seed=3)

    def value(x, w):
        x, w = x.double(), w.double()
        return float((x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w * seed.double()).sum())

    grad, gw = sp.add_norm_backward(None, seed, x, w, eps=EPS)
    for i, made in enumerate((grad, gw)):
        way = _draw(torch.float32, *made.shape, seed=10 + i).double()
        h = 1e-6
        up, down = [x.double(), w.double()], [x.double(), w.double()]
        up[i], down[i] = up[i] + h * way, down[i] - h * way
        diff = (value(*up) - value(*down)) / (2 * h)
        assert abs(float((made.double() * way).sum()) - diff) < 1e-4 * max(1.0, abs(diff))


def test_graphs_beside_each_other():
    """The gradient's partial sums: each graph keeps a workspace of its own."""
    sets = []
    for rows, channels in ((3000, 96), (700, 2056)):
        sets.append([_draw(torch.bfloat16, rows, channels, seed=s) for s in range(3)] + [_draw(torch.bfloat16, channels, seed=9)])

    def run(s):
        h, y = sp.add_norm(s[0], s[1], s[3])
        return (h, y, *sp.add_norm_backward(s[2], y, h, s[3]))

    graphs = []
    for s in sets:
        run(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made = run(s)
        graphs.append((g, made))
    for turn in range(4):
        for s in sets:
            s[0].copy_(_draw(torch.bfloat16, *s[0].shape, seed=20 + turn))
        for g, _ in graphs:
            g.replay()
        sp.add_norm_backward(None, _draw(torch.bfloat16, 50, 4096, seed=1), _draw(torch.bfloat16, 50, 4096, seed=2),
                             _draw(torch.bfloat16, 4096, seed=3))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, (_, made) in zip(sets, graphs):
            assert all(torch.equal(p, q) for p, q in zip(made, run(s)))


def test_refusals():
    x, w = _draw(torch.float16, 10, 48, seed=1), _draw(torch.float16, 48, seed=2)
    bad = [lambda: sp.add_norm(x, x[:5], w), lambda: sp.add_norm(x, x.float(), w), lambda: sp.add_norm(x, None, w.float()),
           lambda: sp.add_norm(x, None, w[:40]), lambda: sp.add_norm(x[:, :12], None, w[:12].contiguous()),
           lambda: sp.add_norm(x, None, w, eps=-1.0), lambda: sp.add_norm(x, None, w, eps=float("nan")),
           lambda: sp.add_norm(x, None, w, out=(x.clone(), x)), lambda: sp.add_norm(x, x.clone(), w, out=(None, x)),
           lambda: sp.add_norm(x.cpu(), None, w.cpu()), lambda: sp.add_norm(x[:1].expand(10, 48), None, w),
           lambda: sp.add_norm(x, x.clone(), w, out=(x, x)), lambda: sp.add_norm(x.t(), None, w),
           lambda: sp.add_norm_backward(None, x, x, w, grad=x), lambda: sp.add_norm_backward(x[:5], x, x, w),
           lambda: sp.add_norm_backward(None, x[:5], x, w), lambda: sp.add_norm(x.reshape(-1)[4:4 + 9 * 48].view(9, 48), None, w)]
    for i, call in enumerate(bad):
        with pytest.raises(sp.SpconvError):
            call()
            pytest.fail(f"call {i} was not refused")
