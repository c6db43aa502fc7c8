"""The precision of the row norm's factor and of its weight gradient in fp32."""
import math

import pytest
import torch

import submanifold_sparse_convolution_device_amd as sp
from linear_reference import UNIT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("channels", [8, 96, 128, 520, 2056, 8192])
def test_factor_of_a_row(channels):
    """Rows of one power of two: their squares and the mean are exact, and y is
    the factor r = 1 / sqrt(h^2 + eps) times that power, exactly.  The
    argument's one rounding, 2^-24 of it, is half of that in r, and r is
    rounded once: 1.5 x 2^-24 of it, and a hundredth for what the products of
    roundings leave."""
    powers = torch.arange(-14, 3, device="cuda", dtype=torch.float32)
    h = torch.exp2(powers)[:, None].expand(-1, channels).contiguous()
    ones = torch.ones(channels, device="cuda")
    for i in range(40):
        eps = float(torch.tensor(1e-6 * 1.37 ** i, dtype=torch.float32))
        _, y = sp.add_norm(h, None, ones, eps=eps)
        assert bool((y == y[:, :1]).all())
        r = 1 / torch.sqrt(h.double().square() + eps)
        far = (y.double() / (h.double() * r) - 1).abs().max()
        assert float(far) <= 1.51 * UNIT, (eps, float(far) / UNIT)


def test_factor_at_the_ends():
    """Rows below and above what the squares' range holds keep their limits."""
    w = torch.ones(8, device="cuda")
    for value, eps, want in ((0.0, 0.0, math.nan), (0.0, 1e-6, 0.0), (2.0 ** -70, 0.0, 1.0), (2.0 ** -62, 0.0, 1.0), (2.0 ** 60, 0.0, 1.0),
                             (2.0 ** 62, 0.0, 1.0), (1e30, 0.0, 0.0), (math.inf, 0.0, math.nan), (math.nan, 0.0, math.nan)):
        _, y = sp.add_norm(torch.full((3, 8), value, device="cuda"), None, w, eps=eps)
        if math.isnan(want):
            assert bool(y.isnan().all()), value
        else:
            # (squares below the normal range keep few bits: 2^-140 has 9)
            assert bool(((y - want).abs() <= (2.0 ** -8 if value == 2.0 ** -70 else 2.0 ** -22)).all()), (value, y[0, 0].item())


@pytest.mark.parametrize("rows,channels", [(100003, 96), (24001, 1024), (400000, 32)])
def test_weight_gradient_sums(rows, channels):
    """The rms error of the weight gradient, in roundings: one leaves 0.425 x
    2^-24 of a value in the mean (uniform in a step, over the steps' places
    between two powers of two).  Terms of either sign add up to the root of
    the sum of their squares, which measures the error: a chain of m additions
    leaves the mean error of (m + 1) / 2 roundings of its sum.  The rows of one
    lane are a chain of at most 13 (100003 rows by 512 workgroups of 16, 24001
    by 512 of 4, 400000 by 1024 of 32), 7 roundings; a term's product and its
    row's factor 2.5; a workgroup's sum and the last one, each rounded from 64
    bits, 2: 11.5.  22 allowed, as the error of 32 columns is 11.5 +- 2.9."""
    g = torch.Generator(device="cuda").manual_seed(7)
    h, gy = (torch.randn(rows, channels, generator=g, device="cuda") for _ in range(2))
    w = torch.ones(channels, device="cuda")
    _, gw = sp.add_norm_backward(None, gy, h, w)
    x = h.double()
    terms = gy.double() * x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    far = (gw.double() - terms.sum(0)).square().mean().sqrt() / terms.square().sum(0).mean().sqrt()
    roundings = (float(far) / (0.425 * UNIT)) ** 2
    assert roundings <= 22, roundings
