"""Products of rows and the row norm in 64 bits, with bounds on what fp32 sums
and one rounding may leave.

Bounds, elementwise: a sum of k products in fp32 is off by at most (k + 1) /
2^24 of the sum of the products' sizes S (each addition by half a unit of a
partial sum, which S bounds); fp32 operands take six plane products for one
and leave out at most 2^-24 of a product, so 6 k + 2 stands for k + 1.  An
output is rounded once, by at most eps / 2 of its value.
"""
import math

import torch

UNIT = 2.0 ** -24
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# the largest slope of gelu (1.1290) and silu (1.0999)
STEEPEST = 1.13
# an activation in 16-bit types: the tail's fit (1.2e-5 of at most 1/2) and a few units of the
# exponential and reciprocal; in fp32 a few units of the library's functions
ACT_ERROR = {torch.float32: 8 * UNIT, torch.float16: 1e-5, torch.bfloat16: 1e-5}


def rounding(dtype):
    return torch.finfo(dtype).eps / 2


# what an fp16 result below its normal range is off by: half of 2^-24
def smallest(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def sum_error(dtype, k):
    return ((6 * k + 2 if dtype == torch.float32 else k + 1) + 2) * UNIT


def act(name, z):
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def groups_of(cu, rows, groups):
    """(group, first row, end) of every group; dense: the whole batch."""
    if cu is None:
        return [(0, 0, rows)]
    b = [min(max(int(v), 0), rows) for v in cu.tolist()]
    return [(e, b[e], b[e + 1]) for e in range(groups)]


def product(x, w, cu=None, transposed=False):
    """(x W, |x| |W|) over rows or groups of rows, zeros for rows of none."""
    w = w.double().reshape(-1, *w.shape[-2:])
    if transposed:
        w = w.transpose(1, 2).contiguous()
    x = x.double()
    out = x.new_zeros(x.shape[0], w.shape[2])
    size = torch.zeros_like(out)
    for e, lo, hi in groups_of(cu, x.shape[0], w.shape[0]):
        if hi > lo:
            out[lo:hi] = x[lo:hi] @ w[e]
            size[lo:hi] = x[lo:hi].abs() @ w[e].abs()
    return out, size


def weight_gradients(x, grad, groups, cu=None):
    """(x^T grad, |x|^T |grad|, sums of grad, of |grad|) of every group."""
    x, grad = x.double(), grad.double()
    made = []
    for _, lo, hi in groups_of(cu, x.shape[0], groups):
        a, g = x[lo:max(lo, hi)].t().contiguous(), grad[lo:max(lo, hi)]
        made.append((a @ g, a.abs() @ g.abs(), g.sum(0), g.abs().sum(0)))
    return [torch.stack(t) for t in zip(*made)]


def row_of_group(cu, rows, groups, device):
    """Whether each row is of a group."""
    there = torch.zeros(rows, dtype=torch.bool, device=device)
    for _, lo, hi in groups_of(cu, rows, groups):
        there[lo:hi] = True
    return there


def close(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, what
    far = (got - ref).abs()
    ok = (far <= bound) | (got == ref)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off, first at {i}: {float(got.flatten()[i])} "
                             f"for {float(ref.flatten()[i])}, bound {float(bound.expand_as(ref).flatten()[i])}")
