"""Products of rows and their gradients over small whole numbers: every sum
stays below 2^24, so fp32 holds it exactly in any order, and each result has
to be the 64-bit one rounded once.  A part, a tail or a row left out or
counted twice shows, however long the sum."""
import pytest
import torch

import submanifold_sparse_convolution_device_amd as sp
from linear_reference import DTYPES, groups_of, product, row_of_group, weight_gradients
from test_gpu_linear import GROUPS, SIZES, _offsets

pytestmark = pytest.mark.gpu

# rows, c_in, c_out, lengths of the groups: the larger tiles, whole rounds and
# the rows after them, parts of long groups, many tiles a group, few rows
LARGE = [(12900, 584, 1032, None), (13057, 584, 1031, None), (13057, 1032, 584, None), (70, 4000, 4104, None),
         (20011, 128, 192, None), (65537, 1024, 256, None), (140011, 256, 200, None), (90011, 520, 500, None),
         (140011, 256, 200, [100001, 0, 9, 40000]), (90011, 520, 500, [50001, 0, 9, 40000]), (35424, 40, 48, [20000, 0, 1, 3001, 0, 12345]),
         (1219, 1000, 328, [1, 0, 700, 3, 90, 0, 0, 2, 400]), (6021, 1000, 328, [0, 1, 5800, 199]), (6021, 1000, 328, [5000, 0, 1000]),
         (5120, 1032, 512, [40] * 128), (2000, 512, 1032, [0, 900, 1, 1000, 0, 0] + [3] * 33), (128, 3000, 2056, None),
         (8000, 256, 256, [0] * 40 + [8000] + [0] * 23), (200000, 512, 512, [12500] * 16), (300, 1024, 33000, None)]


def _whole(dtype, *shape, seed, most=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def _forward(x, w, b, residual, cu):
    dtype, rows = x.dtype, x.shape[0]
    out, pre = sp.linear(x, w, b, activation="relu", residual=residual, cu=cu, return_pre=True)
    z, size = product(x, w, cu)
    assert float(size.max()) < 2 ** 23
    for e, lo, hi in groups_of(cu, rows, 1 if cu is None else w.shape[0]):
        z[lo:hi] += (b if cu is None else b[e]).double()
    there = torch.ones(rows, 1, device="cuda") if cu is None else row_of_group(cu, rows, w.shape[0], "cuda")[:, None]
    assert torch.equal(pre, z.to(dtype)), "pre"
    assert torch.equal(out, (z.clamp(min=0) + residual.double() * there).to(dtype)), "out"


def _backward(x, w, grad, before, cu, **rest):
    dtype = x.dtype
    gx, gw, gb = sp.linear_backward(grad, x, w, pre=before, activation="relu", cu=cu, **rest)
    ref, size = product(grad, w, cu, transposed=True)
    assert float(size.max()) < 2 ** 24
    assert torch.equal(gx, (ref * (before > 0)).to(dtype)), "grad_x"
    rw, sw, rb, _ = weight_gradients(x, grad, 1 if cu is None else w.shape[0], cu)
    assert float(sw.max()) < 2 ** 24
    assert torch.equal(gw.double().reshape(rw.shape), rw), "grad_weight"
    assert torch.equal(gb.double().reshape(rb.shape), rb), "grad_bias"
    return gx, gw, gb


def _case(dtype, rows, c_in, c_out, groups, seed):
    lead = () if groups is None else (groups,)
    return (_whole(dtype, rows, c_in, seed=seed), _whole(dtype, *lead, c_in, c_out, seed=seed + 1, most=2),
            _whole(dtype, *lead, c_out, seed=seed + 2, most=50), _whole(dtype, rows, c_out, seed=seed + 3, most=50))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,c_in,c_out", SIZES)
def test_sizes(dtype, rows, c_in, c_out):
    x, w, b, residual = _case(DTYPES[dtype], rows, c_in, c_out, None, 10)
    _forward(x, w, b, residual, None)
    _backward(x, w, _whole(x.dtype, rows, c_out, seed=20), _whole(x.dtype, rows, c_in, seed=21), None)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lengths", GROUPS)
@pytest.mark.parametrize("c_in,c_out", [(64, 96), (31, 5), (136, 320), (520, 72)])
def test_groups(dtype, lengths, c_in, c_out):
    rows = sum(lengths) + 40
    cu = _offsets(lengths, 3)
    x, w, b, residual = _case(DTYPES[dtype], rows, c_in, c_out, len(lengths), 30)
    _forward(x, w, b, residual, cu)
    _backward(x, w, _whole(x.dtype, rows, c_out, seed=40), _whole(x.dtype, rows, c_in, seed=41), cu)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("at", range(len(LARGE)))
def test_large(dtype, at):
    rows, c_in, c_out, lengths = LARGE[at]
    cu = None if lengths is None else _offsets(lengths)
    x, w, b, residual = _case(DTYPES[dtype], rows, c_in, c_out, None if lengths is None else len(lengths), 50)
    _forward(x, w, b, residual, cu)
    _backward(x, w, _whole(x.dtype, rows, c_out, seed=60), _whole(x.dtype, rows, c_in, seed=61), cu)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("pad", [16, 3])
def test_slices(dtype, pad):
    """Slices of wider rows, aligned and not."""
    dt, rows, c_in, c_out = DTYPES[dtype], 30011, 72, 136
    skip = 8 if pad == 16 else 0
    x = _whole(dt, rows, c_in + pad, seed=70)[:, skip:skip + c_in]
    _, w, b, _ = _case(dt, 1, c_in, c_out, None, 71)
    _forward(x, w, b, _whole(dt, rows, c_out + pad, seed=72, most=50)[:, pad:], None)
    into = torch.empty(rows, c_in + pad, dtype=dt, device="cuda")[:, pad:]
    _backward(x, w, _whole(dt, rows, c_out + 16, seed=73)[:, 8:8 + c_out], _whole(dt, rows, c_in + pad, seed=74)[:, pad:], None, grad_x=into)


def test_far_rows():
    """The weight gradient over more than 2^31 elements of grad_out."""
    rows, c_in, c_out = 2_200_000, 8, 1000
    x = _whole(torch.bfloat16, rows, c_in, seed=80)
    grad = _whole(torch.bfloat16, rows, c_out, seed=81, most=2)
    _, gw, gb = sp.linear_backward(grad, x, _whole(torch.bfloat16, c_in, c_out, seed=82), inputs=False)
    rw, rb = torch.zeros(c_in, c_out, dtype=torch.float64, device="cuda"), torch.zeros(c_out, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 100_000):
        g = grad[lo:lo + 100_000].double()
        rw += x[lo:lo + 100_000].t().contiguous().double() @ g
        rb += g.sum(0)
    assert torch.equal(gw.double(), rw) and torch.equal(gb.double(), rb)


@pytest.mark.parametrize("rows,c_in,c_out,lengths", [(9, 48, 40, None), (30011, 72, 131, None), (30011, 64, 96, [20000, 0, 10000]), (300, 64, 96, [100] * 3)])
def test_weight_gradient_without_the_bias(rows, c_in, c_out, lengths):
    """grad_bias NULL, a choice of the C call alone: the weights' gradient is
    the same, one part and several, and no sums are written."""
    cu = None if lengths is None else _offsets(lengths)
    groups = 1 if lengths is None else len(lengths)
    x, w, _, grad = _case(torch.float16, rows, c_in, c_out, None if lengths is None else groups, 90)
    _, want, _ = sp.linear_backward(grad, x, w, cu=cu, inputs=False)
    got = torch.full(w.shape, float("nan"), dtype=torch.float32, device="cuda")
    args = sp.spconv_linear(x=x.data_ptr(), weight=w.data_ptr(), cu=0 if cu is None else cu.data_ptr(), x_row_stride=c_in, rows=rows,
                            groups=groups, c_in=c_in, c_out=c_out, activation=0, dtype=1)
    grads = sp.spconv_linear_gradients(grad_out=grad.data_ptr(), grad_weight=got.data_ptr(), grad_out_row_stride=c_out)
    sp.spconv_linear_backward(args, grads, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(got, want)
