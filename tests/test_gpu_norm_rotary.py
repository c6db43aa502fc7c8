"""The head norm with the position rotation on the GPU against the 64-bit
reference (bounds derived in attention_reference.py)."""
import math

import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


def _near(name, got, want, tol):
    got = got.double().cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaN at other places"
    diff = torch.where(nan, 0.0, got - torch.where(nan, 0.0, want)).abs()
    tol = torch.where(torch.isnan(tol), 0.0, tol)
    assert bool((diff <= tol).all()), f"{name}: |err| {float(diff.max()):.3e}, at most {float((diff / tol.clamp(min=1e-300)).max()):.2f} times its bound"


def _table(extent, pairs, base=100.0):
    angle = torch.arange(extent, dtype=torch.float64)[:, None] * base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def _case(seed, rows, heads, kv_heads, dim, dtype, axes, rotary, extent=300):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    x = (torch.randn(rows, heads + 2 * kv_heads, dim, generator=g) * 2).to(dt)
    w = (1 + 0.3 * torch.randn(2, dim, generator=g)).to(dt)
    grads = torch.randn(rows, heads + kv_heads, dim, generator=g).to(dt)
    positions = torch.randint(0, extent, (rows, axes), generator=g, dtype=torch.int32)
    table = _table(extent, rotary // (2 * axes)) if rotary else None
    return x, w, grads, positions, table


def _check(sp, x, w, grads, positions, table, heads, kv_heads, rotary, interleaved, eps=1e-6, weights=(True, True)):
    xd, wd, gd = x.to(DEV), w.to(DEV), grads.to(DEV)
    h = {"rotary_dim": rotary, "interleaved": interleaved, "eps": eps}
    td = None if table is None else table.to(DEV)
    pd = positions.to(DEV)
    qw, kw = (wd[i] if weights[i] else None for i in (0, 1))
    args = (xd[:, :heads], xd[:, heads:heads + kv_heads], qw, kw, td, pd)
    print(f"[norm_rotary] {x.dtype} {tuple(x.shape)} heads {heads}/{kv_heads} axes {positions.shape[1]} rotary {rotary} "
          f"interleaved {interleaved}", flush=True)
    out = sp.norm_rotary(*args, **h)
    back = sp.norm_rotary_backward(gd[:, :heads], gd[:, heads:], *args, **h)
    for i, (a, b, go) in enumerate(((0, heads, grads[:, :heads]), (heads, heads + kv_heads, grads[:, heads:]))):
        want = ref.norm_rotary(x[:, a:b], w[i] if weights[i] else None, table, positions, rotary, interleaved, eps, go)
        _near(f"out {i}", out[i], want["out"], want["out_tol"])
        _near(f"grad {i}", back[i], want["grad"], want["grad_tol"])
        if weights[i]:
            _near(f"grad_weight {i}", back[2 + i], want["grad_weight"], want["grad_weight_tol"])
        else:
            assert back[2 + i] is None
    return out, back


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,axes,rotary", [(8, 1, 8), (8, 3, 6), (16, 3, 12), (24, 2, 16), (32, 3, 24), (40, 3, 36), (48, 1, 30),
                                             (64, 3, 60), (64, 1, 32), (72, 4, 56), (96, 3, 96), (120, 1, 120), (128, 1, 64),
                                             (128, 3, 126), (128, 1, 128), (32, 1, 2)])
def test_head_sizes_axes_and_layouts(sp, dtype, interleaved, dim, axes, rotary):
    c = _case(dim + axes, 75, 3, 2, dim, dtype, axes, rotary)
    _check(sp, *c, 3, 2, rotary, interleaved)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 31, 64, 257, 4001])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (16, 2)])
def test_rows_and_heads(sp, dtype, rows, heads, kv_heads):
    c = _case(rows, rows, heads, kv_heads, 32, dtype, 3, 24)
    _check(sp, *c, heads, kv_heads, 24, False)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_norm_alone_rotation_alone_and_neither(sp, dtype):
    c = _case(1, 50, 4, 2, 48, dtype, 1, 48)
    _check(sp, *c[:4], None, 4, 2, 0, False)
    _check(sp, *c, 4, 2, 48, True, weights=(False, False))
    _check(sp, *c, 4, 2, 48, False, weights=(True, False))
    x = c[0].to(DEV)
    q, k = sp.norm_rotary(x[:, :4], x[:, 4:6])
    assert torch.equal(q, x[:, :4]) and torch.equal(k, x[:, 4:6])


def test_one_tensor_only(sp):
    x, w, grads, positions, table = _case(2, 40, 3, 2, 64, "bf16", 1, 64)
    xd, wd, td, pd, gd = (t.to(DEV) for t in (x, w, table, positions, grads))
    both = sp.norm_rotary(xd[:, :3], xd[:, 3:5], wd[0], wd[1], td, pd)
    q, none = sp.norm_rotary(xd[:, :3], None, wd[0], None, td, pd)
    assert none is None and torch.equal(q, both[0])
    none, k = sp.norm_rotary(None, xd[:, 3:5], None, wd[1], td, pd[:, 0])
    assert none is None and torch.equal(k, both[1])
    full = sp.norm_rotary_backward(gd[:, :3], gd[:, 3:], xd[:, :3], xd[:, 3:5], wd[0], wd[1], td, pd)
    part = sp.norm_rotary_backward(None, gd[:, 3:], None, xd[:, 3:5], None, wd[1], td, pd)
    assert part[0] is None and part[2] is None
    assert torch.equal(part[1], full[1]) and torch.equal(part[3], full[3])


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_into_slices(sp, interleaved):
    """Outputs over their inputs, gradients over the outputs' gradients, and
    coordinates read from [N, 4] rows."""
    x, w, grads, positions, table = _case(3, 333, 4, 4, 32, "bf16", 3, 24)
    coords = torch.cat([torch.full((333, 1), 9999, dtype=torch.int32), positions], 1).to(DEV)
    xd, wd, td, gd = (t.to(DEV) for t in (x, w, table, grads))
    h = dict(interleaved=interleaved)
    want = sp.norm_rotary(xd[:, :4], xd[:, 4:8], wd[0], wd[1], td, positions.to(DEV), **h)
    wback = sp.norm_rotary_backward(gd[:, :4], gd[:, 4:], xd[:, :4], xd[:, 4:8], wd[0], wd[1], td, positions.to(DEV), **h)
    back = sp.norm_rotary_backward(gd[:, :4], gd[:, 4:], xd[:, :4], xd[:, 4:8], wd[0], wd[1], td, coords[:, 1:],
                                   grads=(gd[:, :4], gd[:, 4:]), **h)
    for a, b in zip(back, wback):
        assert torch.equal(a, b)
    v = xd[:, 8:].clone()
    got = sp.norm_rotary(xd[:, :4], xd[:, 4:8], wd[0], wd[1], td, coords[:, 1:], out=(xd[:, :4], xd[:, 4:8]), **h)
    assert torch.equal(got[0], want[0]) and torch.equal(xd[:, 4:8], want[1]) and torch.equal(xd[:, 8:], v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_outside_the_table(sp, interleaved):
    """Their axis' pairs are NaN; nothing else is, and nothing is read there."""
    x, w, grads, positions, table = _case(4, 60, 2, 2, 32, "f32", 3, 24)
    positions[3, 0], positions[10, 1], positions[11, 2], positions[59, 0] = -1, 300, 2 ** 31 - 1, -2 ** 31
    xd, wd, td = x.to(DEV), w.to(DEV), table.to(DEV)
    q, k = sp.norm_rotary(xd[:, :2], xd[:, 2:4], wd[0], wd[1], td, positions.to(DEV), interleaved=interleaved)
    for i, got in enumerate((q, k)):
        want = ref.norm_rotary(x[:, 2 * i:2 * i + 2], w[i], table, positions, 24, interleaved, 1e-6)
        _near("out", got, want["out"], want["out_tol"])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_zero_rows_and_extreme_values(sp, dtype):
    """Rows of zeros (eps holds them), of the smallest and of large values."""
    x, w, grads, positions, table = _case(5, 12, 2, 1, 16, dtype, 1, 16)
    x[0] = 0
    x[1] = 6e-5
    x[2] = 250.0
    _check(sp, x, w, grads, positions, table, 2, 1, 16, False, eps=1e-3)
    no_rows = x[:0].to(DEV)
    q, k = sp.norm_rotary(no_rows[:, :2], no_rows[:, 2:3], w[0].to(DEV), w[1].to(DEV))
    assert q.shape == (0, 2, 16) and k.shape == (0, 1, 16)
    got = sp.norm_rotary_backward(q, k, q, k, w[0].to(DEV), w[1].to(DEV))
    assert bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_table_of_angles(sp):
    for extent, pairs, base, scale in ((1, 1, 10000.0, 1.0), (700, 12, 10000.0, 1.0), (5000, 4, 100.0, 0.25), (65536, 64, 5e5, 1.0)):
        got = sp.rotary_table(extent, pairs, base, scale, device=DEV).double().cpu()
        p = torch.arange(extent, dtype=torch.float64)[:, None]
        angle = p * scale * base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        want = torch.stack([angle.cos(), angle.sin()], -1)
        # fp32's rounding, and 64-bit roundings of the angle
        assert bool(((got - want).abs() <= 2.0 ** -25 + 1e-15 * extent).all())


def test_same_bits_and_another_stream(sp):
    x, w, grads, positions, table = _case(6, 5000, 4, 2, 64, "bf16", 1, 64)
    xd, wd, td, pd, gd = (t.to(DEV) for t in (x, w, table, positions, grads))

    def step():
        a = (xd[:, :4], xd[:, 4:6], wd[0], wd[1], td, pd)
        return (*sp.norm_rotary(*a), *sp.norm_rotary_backward(gd[:, :4], gd[:, 4:], *a))

    first = step()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        second = step()
    third = step()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_gradients_against_differences(sp):
    x, w, grads, positions, table = _case(7, 9, 2, 1, 24, "f32", 3, 18)
    args = [t.to(DEV) for t in (x, w, table, positions, grads)]
    got = sp.norm_rotary_backward(args[4][:, :2], args[4][:, 2:], args[0][:, :2], args[0][:, 2:3], args[1][0], args[1][1], args[2], args[3])
    g = torch.Generator().manual_seed(1)
    tol = ref.norm_rotary(x[:, :2], w[0], table, positions, 18, False, 1e-6, grads[:, :2])
    h = 1e-5
    for name, at in (("grad", 0), ("grad_weight", 2)):
        base = (x[:, :2].double(), w[0].double())
        u = torch.randn(base[at // 2].shape, generator=g, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            xs, ws = (b + sign * h * u if i == at // 2 else b for i, b in enumerate(base))
            y = xs / torch.sqrt((xs * xs).mean(-1, keepdim=True) + 1e-6) * ws
            c, s = ref.turn_factors(table, positions, 18)
            z = torch.cat([y[..., :9] * c - y[..., 9:18] * s, y[..., :9] * s + y[..., 9:18] * c, y[..., 18:]], -1)
            ends.append(float((z * grads[:, :2].double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        mine = float((got[at].double().cpu() * u).sum())
        assert abs(mine - slope) <= float((tol[name + "_tol"] * u.abs()).sum()) + 1e-6 * (1 + abs(slope)), name


def test_refusals(sp):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, k, w = torch.zeros(10, 4, 32, **bf), torch.zeros(10, 2, 32, **bf), torch.ones(32, **bf)
    table, pos = torch.zeros(8, 16, 2, device=DEV), torch.zeros(10, dtype=torch.int32, device=DEV)

    def status(*a, **kw):
        with pytest.raises(sp.SpconvError) as e:
            sp.norm_rotary(*a, **kw)
        return e.value.name

    assert status(q.double(), k.double()) == "SPCONV_ERR_UNSUPPORTED"
    assert status(torch.zeros(10, 4, 12, **bf), torch.zeros(10, 4, 12, **bf)) == "SPCONV_ERR_UNSUPPORTED"
    assert status(torch.zeros(10, 4, 136, **bf), torch.zeros(10, 4, 136, **bf)) == "SPCONV_ERR_UNSUPPORTED"
    for bad, kw in (((None, None), {}), ((q, k[:9], w, w, table, pos), {}), ((q, k.float(), w, w, table, pos), {}),
                    ((q, k, w[:16], w, table, pos), {}), ((q, k, w.float(), w, table, pos), {}), ((q, k, w, w, table, None), {}),
                    ((q, k, w, w, table, pos.long()), {}), ((q, k, w, w, table, pos[:9]), {}), ((q, k, w, w, table.half(), pos), {}),
                    ((q, k, w, w, table.cpu(), pos), {}), ((q, k, w, w, table, pos), {"rotary_dim": 16}),
                    ((q, k, w, w, None, pos), {"rotary_dim": 32}), ((q, k, w, w), {"eps": -1.0}), ((q, k, w, w), {"eps": math.nan}),
                    ((q, k, w, w), {"out": (q, q[:, :2])}), ((q, k, w, w), {"out": (q.transpose(0, 1), k)}),
                    ((q, k, w, w, torch.zeros(8, 32, 2, device=DEV), pos), {}),
                    ((q, k, w, w, table, torch.zeros(10, 5, dtype=torch.int32, device=DEV)), {})):
        assert status(*bad, **kw) == "SPCONV_ERR_INVALID_ARG"
