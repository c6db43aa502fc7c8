"""Values of the activations inside the products of rows, seen past the rounding
of the output: a residual that cancels the activation leaves its error."""
import math

import pytest
import torch

import submanifold_sparse_convolution_device_amd as sp
from linear_reference import DTYPES, UNIT, act, rounding, smallest

pytestmark = pytest.mark.gpu


def _one(dtype, z, activation, residual=None):
    """activation(z) + residual of single values, through products by 1."""
    eye = torch.ones(1, 1, dtype=dtype, device="cuda")
    return sp.linear(z[:, None].contiguous(), eye, activation=activation, residual=None if residual is None else residual[:, None].contiguous())[:, 0]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gelu_below_its_rounding(dtype):
    """gelu is z less |z| times the normal distribution's lower tail at -|z|,
    or that product alone.  The tail's fit is off by 4.7e-6 of it.  Up to
    |z| = 4 the exponential's argument is at most 11.6 (in powers of two) and
    rounded twice and by its constant, 2.5 x 2^-24 of it: 1.2e-6 of the
    result; the exponential, the reciprocal, the polynomial and the products
    are off by a unit of 2^-23 each at most, ten of them 1.2e-6: 7.1e-6 of the
    tail's product in all.  The difference and the addition of the residual
    round by 2^-24 of z and of the residual, the output once."""
    dt = DTYPES[dtype]
    z = torch.cat([torch.linspace(-4, 4, 20001), torch.logspace(-3, 0, 2000), -torch.logspace(-3, 0, 2000)]).to(dt).cuda()
    ref = act("gelu", z.double())
    residual = (-ref).to(dt)
    got = _one(dt, z, "gelu", residual).double()
    want = ref + residual.double()
    below = z.double().abs() * 0.5 * torch.erfc(z.double().abs() / math.sqrt(2))
    bound = 7.1e-6 * below + UNIT * (z.double().abs() + residual.double().abs())
    bound = bound + rounding(dt) * (want.abs() + bound) + smallest(dt)
    over = (got - want).abs() / bound
    assert float(over.max()) <= 1, f"{float(over.max())} of the bound at z = {float(z[over.argmax()])}"


@pytest.mark.parametrize("rows", [6, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("activation", ["relu", "silu", "gelu"])
def test_infinite_sums_with_a_residual(dtype, activation, rows):
    """The activation of an infinite sum is infinite (or 0) when the residual
    is added, whatever its size, in each of the products: few rows (6 and, by
    parts of a long contraction, 1), tiles, and weights in registers."""
    dt = DTYPES[dtype]
    big = torch.finfo(dt).max
    inf = math.inf
    for c_in, c_out in ((8, 64), (8, 7), (2048, 64), (600, 64)):
        x = torch.zeros(rows, c_in, dtype=dt, device="cuda")
        x[:, 0] = torch.tensor([inf, inf, inf, -inf, inf, 1.0], dtype=dt).cuda().repeat(rows // 6)
        w = torch.zeros(c_in, c_out, dtype=dt, device="cuda")
        w[0] = 1
        residual = torch.tensor([-big, -inf, inf, 5.0, 0.0, -big], dtype=dt).cuda().repeat(rows // 6)[:, None].expand(rows, c_out).contiguous()
        for place in (None, residual.clone()):
            res = residual if place is None else place
            got, pre = sp.linear(x, w, activation=activation, residual=res, out=place, return_pre=True)
            assert bool((pre[0::6] == inf).all()) and bool((pre[3::6] == -inf).all())
            for at, want in ((0, inf), (2, inf), (3, 5.0), (4, inf), (5, -big)):
                assert bool((got[at::6] == want).all()), (c_in, c_out, at, got[at, 0].item())
            assert bool(got[1::6].isnan().all()), (c_in, c_out, got[1, 0].item())
        one = sp.linear(x[:1], w, activation=activation, residual=residual[:1])
        assert bool((one == inf).all())


def test_fp32_gelu_keeps_its_lower_tail():
    """Relative bounds down to z = -12, where gelu is -2e-32.  The error
    function's argument z / sqrt 2 is off by 1.3 x 2^-24 of it (the constant's
    rounding and the product's), which changes a tail exp(-z^2 / 2) / |z| by
    1.3 (z^2 + 1) / 2^24 of it; the exponential's argument by 2 roundings, z^2
    / 2^24.  The library's functions may be off by 16 units of 2^-23 (erfc)
    and 3 (exp), a product or sum by a rounding."""
    z = torch.cat([torch.linspace(-12, 12, 40001), -torch.logspace(-4, 0, 1000)]).float().cuda()
    zd = z.double()
    phi = 0.5 * torch.erfc(-zd / math.sqrt(2))
    ref = zd * phi
    share = (1.3 * (zd * zd + 1) * (zd < 0) + 1.3 * (zd >= 0) + 36) * UNIT
    got = _one(torch.float32, z, "gelu").double()
    over = (got - ref).abs() / (share * ref.abs() + 1e-300)
    assert float(over.max()) <= 1, f"value: {float(over.max())} of the bound at z = {float(z[over.argmax()])}"
    bell = zd * torch.exp(-0.5 * zd * zd) / math.sqrt(2 * math.pi)
    got = sp.activation_backward(torch.ones_like(z)[None], z[None], "gelu")[0].double()
    over = (got - (phi + bell)).abs() / (share * phi + (zd * zd + 12) * UNIT * bell.abs() + UNIT * (phi + bell).abs())
    assert float(over.max()) <= 1, f"slope: {float(over.max())} of the bound at z = {float(z[over.argmax()])}"
