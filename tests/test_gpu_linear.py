"""Products of rows with their epilogue, over one batch and over groups, and
their gradients, against the formulas in 64 bits."""
import math

import pytest
import torch

import submanifold_sparse_convolution_device_amd as sp
from linear_reference import (ACT_ERROR, DTYPES, STEEPEST, UNIT, act, close, groups_of, product, rounding, row_of_group, slope,
                              smallest, sum_error, weight_gradients)

pytestmark = pytest.mark.gpu

# rows, c_in, c_out: one row, tiles' edges, lengths that are no whole pieces,
# few and many columns, few rows by a long contraction, single values
SIZES = [(1, 8, 8), (1, 2048, 264), (5, 20, 19), (33, 64, 64), (64, 96, 20), (127, 40, 136), (300, 257, 131), (1000, 1, 1),
         (257, 512, 384), (2000, 72, 300), (513, 640, 264), (31, 1000, 33), (4097, 33, 7),
         # contractions short enough for weights in registers, one tile and many of each workgroup
         (40, 16, 64), (300, 256, 136), (1000, 200, 64), (700, 136, 128), (30001, 256, 1024), (333, 128, 72), (40000, 128, 264),
         (20000, 64, 96), (20000, 248, 88)]
GROUPS = [[0, 5, 0, 1, 64, 130, 0], [3] * 70, [1], [0, 0, 0], [700, 1, 129, 0, 40], [0] * 130 + [9, 200] + [0] * 5,
          [3000, 0, 1, 5000, 33, 0, 7000], [150, 0, 0, 31, 400]]


def _draw(dtype, *shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _case(dtype, rows, c_in, c_out, seed, groups=None):
    lead = () if groups is None else (groups,)
    x = _draw(dtype, rows, c_in, seed=seed)
    w = _draw(dtype, *lead, c_in, c_out, seed=seed + 1, scale=c_in ** -0.5)
    b = _draw(dtype, *lead, c_out, seed=seed + 2, scale=0.5)
    return x, w, b


def _offsets(lengths, before=0):
    return torch.tensor([before] + [before + sum(lengths[:i + 1]) for i in range(len(lengths))], dtype=torch.int32, device="cuda")


def _bias_rows(b, cu, rows, c_out):
    if cu is None:
        return b.double().expand(rows, c_out)
    full = torch.zeros(rows, c_out, dtype=torch.float64, device=b.device)
    for e, lo, hi in groups_of(cu, rows, b.shape[0]):
        full[lo:hi] = b[e].double()
    return full


def _check_forward(x, w, b, activation, residual, cu=None, out=None):
    dtype, rows, k, n = x.dtype, x.shape[0], x.shape[1], w.shape[-1]
    keep = residual.clone() if residual is not None else None
    got, pre = sp.linear(x, w, b, activation=activation, residual=residual, cu=cu, out=out, return_pre=True)
    alone = sp.linear(x, w, b, activation=activation, residual=keep, cu=cu)
    assert torch.equal(got, alone) or bool(got.isnan().any())
    z, size = product(x, w, cu)
    if b is not None:
        full = _bias_rows(b, cu, rows, n)
        z, size = z + full, size + full.abs()
    err = sum_error(dtype, k) * size
    close(pre, z, err + rounding(dtype) * z.abs() * (1 + UNIT) + smallest(dtype), "pre")
    ref = act(activation, z)
    bound = STEEPEST * err + ACT_ERROR[dtype] * (z.abs() if activation else 0.0)
    if residual is not None:
        inside = torch.ones(rows, dtype=torch.bool, device=x.device) if cu is None else row_of_group(cu, rows, w.shape[0], x.device)
        ref = ref + keep.double() * inside[:, None]
        bound = bound + UNIT * ref.abs()
    close(got, ref, bound + rounding(dtype) * (ref.abs() + bound) + smallest(dtype), "out")
    return got


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("at", range(len(SIZES)))
def test_forward(dtype, at):
    rows, c_in, c_out = SIZES[at]
    dt = DTYPES[dtype]
    x, w, b = _case(dt, rows, c_in, c_out, 10 * at)
    activation = (None, "relu", "silu", "gelu")[at % 4]
    residual = _draw(dt, rows, c_out, seed=10 * at + 3) if at % 3 else None
    _check_forward(x, w, b if at % 5 else None, activation, residual)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu"])
def test_forward_activations(dtype, activation):
    """Arguments from -12 to 12: the tails of the activations."""
    dt = DTYPES[dtype]
    x = torch.linspace(-12, 12, 4096).to(dt).cuda()[:, None].contiguous()
    w = torch.tensor([[1.0, 0.5, 0.25]], dtype=dt).cuda()
    _check_forward(x, w, torch.zeros(3, dtype=dt).cuda(), activation, None)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("at", range(len(GROUPS)))
def test_forward_groups(dtype, at):
    lengths, dt = GROUPS[at], DTYPES[dtype]
    before, after = (0, 0) if at % 2 else (3, 37)
    rows = before + sum(lengths) + after
    c_in, c_out = [(64, 96), (24, 130), (31, 5), (128, 64), (96, 272), (520, 136), (256, 320), (200, 104)][at]
    if rows == 0:
        rows = 4
    x, w, b = _case(dt, rows, c_in, c_out, 100 + at, len(lengths))
    residual = _draw(dt, rows, c_out, seed=5) if at % 3 == 0 else None
    got = _check_forward(x, w, b, (None, "gelu", "relu")[at % 3], residual, _offsets(lengths, before))
    outside = ~row_of_group(_offsets(lengths, before), rows, len(lengths), x.device)
    assert not bool(got[outside].any())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_large_tiles(dtype):
    """Whole large products: many tiles of the largest shape, ragged edges."""
    dt = DTYPES[dtype]
    x, w, b = _case(dt, 12900, 584, 1032, 7)
    _check_forward(x, w, b, "gelu", _draw(dt, 12900, 1032, seed=1))
    _check_backward(x, w, _draw(dt, 12900, 1032, seed=2))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,c_out", [(13057, 1032), (13057, 1031), (13500, 1032)])
def test_rows_after_whole_rounds(dtype, rows, c_out):
    """One tile's rows more than the largest tiles take in one round."""
    dt = DTYPES[dtype]
    x, w, b = _case(dt, rows, 584, c_out, 8)
    _check_forward(x, w, b, "gelu", _draw(dt, rows, c_out, seed=1))
    x, w, _ = _case(dt, rows, c_out, 584, 8)
    pre = x.clone()
    _check_backward(x[:, :32].contiguous(), w[:32], _draw(dt, rows, 584, seed=2))
    _check_backward(_draw(dt, rows, c_out, seed=3), w, _draw(dt, rows, 584, seed=4), pre=pre, activation="gelu")


def test_rows_after_whole_rounds_in_place():
    """The same with strided rows, the residual in its place, and captured."""
    dt, rows, c_in, c_out = torch.bfloat16, 13061, 1536, 1032
    x = _draw(dt, rows, c_in + 24, seed=1)[:, 16:16 + c_in]
    _, w, b = _case(dt, 8, c_in, c_out, 18)
    wide = _draw(dt, rows, c_out + 40, seed=2)
    kept = wide.clone()
    residual = wide[:, 32:32 + c_out]
    first = _check_forward(x, w, b, "gelu", residual, out=residual).clone()
    assert torch.equal(wide[:, :32], kept[:, :32]) and torch.equal(wide[:, 32 + c_out:], kept[:, 32 + c_out:])
    before = kept[:, 32:32 + c_out].contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        made = sp.linear(x, w, b, activation="gelu", residual=before)
    for turn in range(3):
        made.zero_()
        sp.linear(_draw(dt, 40, 8192, seed=turn), _draw(dt, 8192, 264, seed=9))  # (the stream's workspace in other hands)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(made, first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_sums(dtype):
    """The weight gradient's largest tiles, and weights larger than a tile row."""
    dt = DTYPES[dtype]
    x, w, _ = _case(dt, 70, 4000, 4104, 9)
    _check_backward(x, w, _draw(dt, 70, 4104, seed=2))


def _check_backward(x, w, grad, pre=None, activation=None, cu=None, **rest):
    dtype, rows = x.dtype, x.shape[0]
    groups = 1 if cu is None else w.shape[0]
    gx, gw, gb = sp.linear_backward(grad, x, w, pre=pre, activation=activation, cu=cu, **rest)
    ref, size = product(grad, w, cu, transposed=True)
    bound = sum_error(dtype, w.shape[-1]) * size
    if pre is not None:
        s = slope(activation, pre.double())
        ref, bound = ref * s, STEEPEST * bound + ref.abs() * 4 * ACT_ERROR[dtype] * (1 + pre.double().abs())
    close(gx, ref, bound + rounding(dtype) * (ref.abs() + bound) + smallest(dtype), "grad_x")
    assert gw.dtype == gb.dtype == torch.float32 and gw.shape == w.shape
    rw, sw, rb, sb = weight_gradients(x, grad, groups, cu)
    most = max(hi - lo for _, lo, hi in groups_of(cu, rows, groups))
    close(gw.reshape(rw.shape), rw, sum_error(dtype, most) * sw, "grad_weight")
    close(gb.reshape(rb.shape), rb, (most + 2) * UNIT * sb, "grad_bias")
    return gx, gw, gb


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("at", range(len(SIZES)))
def test_backward(dtype, at):
    rows, c_in, c_out = SIZES[at]
    dt = DTYPES[dtype]
    x, w, _ = _case(dt, rows, c_in, c_out, 200 + at)
    grad = _draw(dt, rows, c_out, seed=300 + at)
    activation = (None, "gelu", "silu", "relu")[at % 4]
    pre = None
    if activation:
        pre = _draw(dt, rows, c_in, seed=400 + at, scale=2.0)
        x = act(activation, pre.double()).to(dt)
    _check_backward(x, w, grad, pre, activation)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("at", range(len(GROUPS)))
def test_backward_groups(dtype, at):
    lengths, dt = GROUPS[at], DTYPES[dtype]
    before, after = (3, 37) if at % 2 else (0, 0)
    rows = max(before + sum(lengths) + after, 2)
    c_in, c_out = [(64, 96), (24, 130), (31, 5), (128, 64), (96, 272), (136, 72), (320, 256), (64, 128)][at]
    x, w, _ = _case(dt, rows, c_in, c_out, 500 + at, len(lengths))
    grad = _draw(dt, rows, c_out, seed=600 + at)
    pre = _draw(dt, rows, c_in, seed=700 + at) if at % 3 == 1 else None
    gx, _, _ = _check_backward(x, w, grad, pre, "gelu" if pre is not None else None, _offsets(lengths, before))
    outside = ~row_of_group(_offsets(lengths, before), rows, len(lengths), x.device)
    assert not bool(gx[outside].any())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_parts_of_groups(dtype):
    """Long groups go by parts of their rows: lengths around the parts' ends,
    an empty group and a group of one row among them."""
    dt = DTYPES[dtype]
    lengths = [20000, 0, 1, 3001, 0, 12345]
    x, w, _ = _case(dt, sum(lengths) + 77, 40, 48, 11, len(lengths))
    _check_backward(x, w, _draw(dt, sum(lengths) + 77, 48, seed=12), cu=_offsets(lengths))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,c_in,c_out", [(140011, 256, 200), (90011, 520, 500)])
@pytest.mark.parametrize("grouped", [False, True])
def test_tiles_of_large_sums(dtype, rows, c_in, c_out, grouped):
    """Weight gradients whose sums go by the larger tiles."""
    dt = DTYPES[dtype]
    lengths = [rows - 40010, 0, 9, 40000]
    x, w, _ = _case(dt, rows, c_in, c_out, 13, len(lengths) if grouped else None)
    _check_backward(x, w, _draw(dt, rows, c_out, seed=14), cu=_offsets(lengths) if grouped else None)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lengths", [[1, 0, 700, 3, 90, 0, 0, 2, 400], [0, 1, 5800, 199], [5000, 0, 1000]])
def test_many_tiles_of_groups(dtype, lengths):
    """Weight gradients of many tiles a group, lengths far apart: one part a
    group, and several."""
    dt = DTYPES[dtype]
    rows = sum(lengths) + 21
    x, w, _ = _case(dt, rows, 1000, 328, 15, len(lengths))
    _check_backward(x, w, _draw(dt, rows, 328, seed=16), cu=_offsets(lengths, 17))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,c_in,c_out,lengths", [
    (37, 4104, 4096, None), (128, 2048, 2056, None), (128, 3000, 2056, None), (40, 4096, 264, [3, 0, 37]),
    (5120, 1032, 512, [40] * 128), (2000, 512, 1032, [0, 900, 1, 1000, 0, 0] + [3] * 33), (700, 2048, 512, [20] * 35)])
def test_rows_by_wavefronts_or_tiles(dtype, rows, c_in, c_out, lengths):
    """Both sides of the choice for few rows of a group."""
    dt = DTYPES[dtype]
    cu = None if lengths is None else _offsets(lengths)
    x, w, b = _case(dt, rows, c_in, c_out, 17, None if lengths is None else len(lengths))
    _check_forward(x, w, b, "silu", _draw(dt, rows, c_out, seed=1), cu)
    _check_backward(x, w, _draw(dt, rows, c_out, seed=2), _draw(dt, rows, c_in, seed=3), "relu", cu)


@pytest.mark.parametrize("rows,c_in,c_out,lengths", [
    (2500, 1032, 500, None), (40011, 40, 264, None), (70001, 264, 57, None), (35000, 300, 64, [0, 20000, 33, 14900])])
def test_fp32_by_64_columns(rows, c_in, c_out, lengths):
    """Tiles of 64 columns, of the product and of both gradients."""
    cu = None if lengths is None else _offsets(lengths)
    x, w, b = _case(torch.float32, rows, c_in, c_out, 19, None if lengths is None else len(lengths))
    _check_forward(x, w, b, "silu", None, cu)
    _check_backward(x, w, _draw(torch.float32, rows, c_out, seed=2), cu=cu)


def test_fp32_is_whole():
    """The rms error of fp32 products: additions leave about sqrt(k) / 2^25 of
    the result's rms, 2^-20 at k = 1024, and twice that is allowed; operands
    without their lowest plane would leave 2^-18.8."""
    x, w, _ = _case(torch.float32, 600, 1000, 260, 21)
    grad = _draw(torch.float32, 600, 260, seed=22)
    gx, gw, _ = sp.linear_backward(grad, x, w)
    pairs = [(sp.linear(x, w), product(x, w)[0]), (gx, product(grad, w, transposed=True)[0]),
             (gw, weight_gradients(x, grad, 1)[0][0])]
    for got, ref in pairs:
        assert float((got.double() - ref).square().mean().sqrt()) <= 2.0 ** -19 * float(ref.square().mean().sqrt())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strides_and_places(dtype):
    """Slices of wider tensors, unaligned rows, the residual in its place, and
    what lies around the outputs left as it was."""
    dt = DTYPES[dtype]
    rows, c_in, c_out = 150, 48, 40
    for pad, skip in ((16, 8), (3, 0)):
        wide = _draw(dt, rows, c_in + pad, seed=1)
        x = wide[:, skip:skip + c_in] if skip else wide[:, :c_in]
        _, w, b = _case(dt, rows, c_in, c_out, 31)
        res = _draw(dt, rows, c_out + pad, seed=2)
        around = res.clone()
        residual = res[:, pad:]
        _check_forward(x, w, b, "silu", residual, out=residual)
        assert torch.equal(res[:, :pad], around[:, :pad])
        grad = _draw(dt, rows, c_out + 16, seed=3)[:, 8:8 + c_out]
        into = _draw(dt, rows, c_in + pad, seed=4)
        around = into.clone()
        pre = _draw(dt, rows, c_in + pad, seed=5)[:, pad:]
        _check_backward(act("gelu", pre.double()).to(dt), w, grad, pre, "gelu", grad_x=into[:, pad:])
        assert torch.equal(into[:, :pad], around[:, :pad])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_parts_of_the_gradients(dtype):
    x, w, _ = _case(DTYPES[dtype], 200, 64, 72, 41)
    grad = _draw(x.dtype, 200, 72, seed=42)
    gx, gw, gb = sp.linear_backward(grad, x, w)
    a, none_w, none_b = sp.linear_backward(grad, x, w, weights=False)
    none_x, b, c = sp.linear_backward(grad, x, w, inputs=False)
    assert none_w is None and none_b is None and none_x is None
    assert torch.equal(a, gx) and torch.equal(b, gw) and torch.equal(c, gb)
    assert sp.linear_backward(grad, x, w, inputs=False, weights=False) == (None, None, None)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_no_rows(dtype):
    dt = DTYPES[dtype]
    x, w, b = _case(dt, 0, 24, 40, 51)
    assert sp.linear(x, w, b, activation="gelu").shape == (0, 40)
    gx, gw, gb = sp.linear_backward(x.new_empty(0, 40), x, w)
    assert gx.shape == (0, 24) and not bool(gw.any()) and not bool(gb.any())
    x, w, b = _case(dt, 0, 24, 40, 52, 3)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert sp.linear(x, w, b, cu=cu).shape == (0, 40)
    gx, gw, gb = sp.linear_backward(x.new_empty(0, 40), x, w, cu=cu)
    assert gw.shape == (3, 24, 40) and not bool(gw.any()) and not bool(gb.any())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_values_that_are_not_finite(dtype):
    """An infinity or NaN reaches its own row, its own column and its own
    group only: not the tile's other rows, nor what lies past an edge."""
    dt = DTYPES[dtype]
    lengths = [70, 0, 45]
    x, w, b = _case(dt, 140, 40, 24, 61, 3)
    cu = _offsets(lengths, 5)
    grad = _draw(dt, 140, 24, seed=62)
    clean = sp.linear(x, w, b, cu=cu)
    gx0, gw0, gb0 = sp.linear_backward(grad, x, w, cu=cu)
    bad = x.clone()
    bad[0], bad[11, 3], bad[75, 39], bad[139] = float("nan"), float("nan"), float("inf"), float("inf")
    out = sp.linear(bad, w, b, cu=cu)
    hit = torch.zeros(140, dtype=torch.bool, device="cuda")
    hit[11] = hit[75] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert bool(out[11].isnan().all()) and not bool(out[75].isfinite().any())
    _, gw, gb = sp.linear_backward(grad, bad, w, cu=cu)
    keep = torch.ones(3, 40, dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[2, 39] = False  # rows 5 .. 74 are group 0, 75 .. 119 group 2
    assert torch.equal(gw[keep], gw0[keep]) and torch.equal(gb, gb0)
    assert bool(gw[0, 3].isnan().all()) and not bool(gw[2, 39].isfinite().any())
    bad = grad.clone()
    bad[2], bad[20, 7] = float("nan"), float("inf")
    gx, gw, gb = sp.linear_backward(bad, x, w, cu=cu)
    hit[:] = False
    hit[20] = True
    assert torch.equal(gx[~hit], gx0[~hit]) and not bool(gx[20].isfinite().any())
    keep = torch.ones(3, 24, dtype=torch.bool, device="cuda")
    keep[0, 7] = False
    assert torch.equal(gb[keep], gb0[keep]) and torch.equal(gw.transpose(1, 2)[keep], gw0.transpose(1, 2)[keep])
    # the epilogue keeps a NaN, also through relu
    z = torch.tensor([[float("nan"), 1.0, -1.0, 0.0]], dtype=dt).cuda()
    eye = torch.eye(1, dtype=dt).cuda()
    got = sp.linear(z.t().contiguous(), eye, activation="relu")
    assert bool(got[0].isnan()) and got[1:, 0].tolist() == [1.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (50, 100), (7, 33)])
def test_activation_backward(dtype, activation, rows, cols):
    dt = DTYPES[dtype]
    pre, grad = _draw(dt, rows, cols, seed=71, scale=4.0), _draw(dt, rows, cols, seed=72)
    pre[0, 0] = 0.0
    got = sp.activation_backward(grad, pre, activation)
    s = slope(activation, pre.double())
    ref = grad.double() * s
    bound = grad.double().abs() * (ACT_ERROR[dt] * (1 + pre.double().abs()) if activation else 0.0)
    close(got, ref, bound + rounding(dt) * (ref.abs() + bound) * (1 + 2 * UNIT) + smallest(dt), "grad_pre")
    # against differences of the activation itself
    h = 1e-6
    diff = (act(activation, pre.double() + h) - act(activation, pre.double() - h)) / (2 * h)
    away = pre.double().abs() > 1e-3  # (relu has a corner)
    assert bool(((s - diff).abs() < 1e-8)[away].all())
    same = grad.clone()
    assert sp.activation_backward(same, pre, activation, out=same) is same and torch.equal(same, got)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("activation,ends,slopes", [
    ("relu", (0.0, math.inf), (0.0, 1.0)), ("silu", (0.0, math.inf), (0.0, 1.0)), ("gelu", (0.0, math.inf), (0.0, 1.0))])
def test_activations_at_the_ends(dtype, activation, ends, slopes):
    """Infinite and largest values take the activation's limits: a stored
    product past fp16's range is infinite, its gradient is not NaN."""
    dt = DTYPES[dtype]
    far = torch.finfo(dt).max
    pre = torch.tensor([-math.inf, -far, -1000.0, 1000.0, far, math.inf, math.nan], dtype=dt).cuda()
    got = sp.activation_backward(torch.ones_like(pre)[None], pre[None], activation)[0].tolist()
    assert got[:6] == [slopes[0]] * 3 + [slopes[1]] * 3
    if activation != "relu":
        assert math.isnan(got[6])
    # an infinite sum in bf16 (the planes of fp32 hold no infinity, and fp16 products cannot reach one)
    top = far if dt == torch.bfloat16 else 2.0 ** 15
    x = torch.tensor([-top, -1000.0, 1000.0, top], dtype=dt).cuda()[:, None]
    w = torch.tensor([[1.0, top if dt == torch.bfloat16 else 1.0]], dtype=dt).cuda()
    out = sp.linear(x, w, activation=activation)
    assert out[:2].abs().max().item() == ends[0]
    assert out[2:, 0].tolist() == x[2:, 0].tolist() and out[3, 1].item() == (ends[1] if dt == torch.bfloat16 else top)


def test_gradient_against_differences():
    """The whole chain in fp32: product, activation, product with residual."""
    x, w1, b1 = _case(torch.float32, 40, 24, 32, 81)
    _, w2, b2 = _case(torch.float32, 40, 32, 24, 82)
    seed = _draw(torch.float32, 40, 24, seed=83)

    def value(x, w1, b1, w2, b2):
        a = act("gelu", x.double() @ w1.double() + b1.double())
        return float(((a @ w2.double() + b2.double() + x.double()) * seed.double()).sum())

    a, pre = sp.linear(x, w1, b1, activation="gelu", return_pre=True)
    out = sp.linear(a, w2, b2, residual=x)
    assert abs(float((out.double() * seed.double()).sum()) - value(x, w1, b1, w2, b2)) < 1e-3
    gpre, gw2, gb2 = sp.linear_backward(seed, a, w2, pre=pre, activation="gelu")
    gx, gw1, gb1 = sp.linear_backward(gpre, x, w1)
    made = (gx + seed, gw1, gb1, gw2, gb2)
    for i, t in enumerate((x, w1, b1, w2, b2)):
        way = _draw(torch.float32, *t.shape, seed=90 + i)
        args = [x.double(), w1.double(), b1.double(), w2.double(), b2.double()]
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        diff = (value(*up) - value(*down)) / (2 * h)
        along = float((made[i].double() * way.double()).sum())
        # fp32 sums of up to 40 x 32 terms of size about 1, and h^2 of the third derivative
        assert abs(along - diff) < 1e-3 * max(1.0, abs(diff)), i


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_same_bits(dtype):
    dt = DTYPES[dtype]
    for rows, c_in, c_out in ((7, 4096, 72), (9000, 64, 48)):
        x, w, b = _case(dt, rows, c_in, c_out, 101)
        grad = _draw(dt, rows, c_out, seed=102)
        first = (sp.linear(x, w, b, activation="silu"), *sp.linear_backward(grad, x, w))
        for _ in range(3):
            again = (sp.linear(x, w, b, activation="silu"), *sp.linear_backward(grad, x, w))
            assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_far_elements():
    """More than 2^31 elements of output: the last rows' places."""
    rows = 2_200_000
    x = _draw(torch.bfloat16, rows, 8, seed=111)
    w = _draw(torch.bfloat16, 8, 1000, seed=112)
    out = sp.linear(x, w)
    for at in (slice(0, 300), slice(rows - 300, rows)):
        ref, size = product(x[at], w)
        close(out[at], ref, sum_error(x.dtype, 8) * size + rounding(x.dtype) * ref.abs() * 1.001, "out")
    gx, gw, _ = sp.linear_backward(out, x, w)
    ref, size = product(out[-300:], w, transposed=True)
    close(gx[-300:], ref, (sum_error(x.dtype, 1000) * size + rounding(x.dtype) * ref.abs()) * 1.001, "grad_x")


def test_offsets_that_break_the_rules():
    """Decreasing, negative and too large offsets: some rows, no fault."""
    x, w, b = _case(torch.float16, 90, 16, 24, 121, 4)
    for cu in ([0, 50, 20, 80, 90], [-5, 10, 20, 30, 1 << 30], [90, 60, 30, 10, 0], [-(1 << 31), 5, (1 << 31) - 1, 7, 7]):
        cu = torch.tensor(cu, dtype=torch.int64).to(torch.int32).cuda()
        assert sp.linear(x, w, b, cu=cu).shape == (90, 24)
        sp.linear_backward(_draw(torch.float16, 90, 24, seed=1), x, w, cu=cu)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ streams and graphs


def _all(x, w, b, grad, cu):
    out, pre = sp.linear(x, w, b, activation="gelu", cu=cu, return_pre=True)
    return (out, pre, sp.activation_backward(grad, pre, "gelu"), *sp.linear_backward(grad, x, w, cu=cu))


@pytest.mark.parametrize("grouped", [False, True])
def test_graphs_beside_each_other(grouped):
    """Captured calls that need workspaces (a long contraction of few rows,
    parts of the rows, copies of odd lengths), replayed in turn with eager
    calls that grow the stream's workspace between."""
    sets = []
    for seed, rows in ((131, 9), (137, 7001)):
        lengths = [rows // 3, 0, rows - rows // 3]
        x, w, b = _case(torch.bfloat16, rows, 1100 if rows < 100 else 41, 67, seed, 3 if grouped else None)
        sets.append((x, w, b, _draw(torch.bfloat16, rows, 67, seed=seed + 4), _offsets(lengths) if grouped else None))
    graphs = []
    for s in sets:
        _all(*s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made = _all(*s)
        graphs.append((g, made))
    for turn in range(4):
        for s in sets:
            s[0].copy_(_draw(torch.bfloat16, *s[0].shape, seed=140 + turn))
        for g, _ in graphs:
            g.replay()
        eager = _case(torch.bfloat16, 3000 * (turn + 1), 100, 99, 150)
        sp.linear_backward(_draw(torch.bfloat16, 3000 * (turn + 1), 99, seed=1), eager[0], eager[1])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, (_, made) in zip(sets, graphs):
            assert all(torch.equal(p, q) for p, q in zip(made, _all(*s)))


def test_two_streams():
    """Calls on two streams at once keep to their own workspaces."""
    sets = [(_case(torch.float16, 11, 3000, 72, 160 + i), _draw(torch.float16, 11, 72, seed=170 + i)) for i in range(2)]
    want = [_all(*c, g, None) for c, g in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    made = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                made[i].append(_all(*sets[i][0], sets[i][1], None))
    torch.cuda.synchronize()
    for i in range(2):
        for got in made[i]:
            assert all(torch.equal(p, q) for p, q in zip(got, want[i]))


def test_refusals_on_the_device():
    x, w, b = _case(torch.float16, 20, 16, 24, 181)
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    bad = [lambda: sp.linear(x, w.float(), b), lambda: sp.linear(x, w, b.float()), lambda: sp.linear(x, w[:8], b),
           lambda: sp.linear(x, w, b, cu=cu), lambda: sp.linear(x, w[None], b[None], cu=cu.long()),
           lambda: sp.linear(x, w[None], b, cu=cu), lambda: sp.linear(x, w[None], b[None], cu=cu[:1]),
           lambda: sp.linear(x, w, b, activation="tanh"), lambda: sp.linear(x.t(), w, b), lambda: sp.linear(x, w.t(), b),
           lambda: sp.linear(x, w, b, residual=x), lambda: sp.linear(x, w, b, out=x.new_empty(20, 16)),
           lambda: sp.linear(x.cpu(), w, b), lambda: sp.linear(x.long(), w, b), lambda: sp.linear(x[0], w, b),
           lambda: sp.linear(x[:1].expand(20, 16), w, b), lambda: sp.linear(x[:, 1:9], w[:8].contiguous(), b),
           lambda: sp.linear_backward(x, x, w), lambda: sp.linear_backward(x.new_empty(20, 24), x, w, pre=x),
           lambda: sp.linear_backward(x.new_empty(20, 24), x, w, activation="gelu"),
           lambda: sp.linear_backward(x.new_empty(20, 24), x, w, grad_x=x),
           lambda: sp.linear(x, w[:, :16].contiguous(), out=x),
           lambda: sp.activation_backward(x, x[:10], "gelu"), lambda: sp.activation_backward(x, x.float(), "gelu"),
           lambda: sp.activation_backward(x, x, "tanh"), lambda: sp.activation_backward(x, x, "gelu", out=x)]
    for i, call in enumerate(bad):
        with pytest.raises(sp.SpconvError):
            call()
            pytest.fail(f"call {i} was not refused")
