"""The block of examples/voxel_transformer.py: its output and gradients against
the same block in 64-bit torch with autograd, and training steps that run."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import voxel_transformer
    return voxel_transformer


def _norm(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _reference(block, e, x, grad):
    """The block in fp64 on the CPU, differentiated by autograd."""
    w = {n: t.bfloat16().double().cpu().requires_grad_() for n, t in block.weights.items()}
    coords = block.coords.cpu().numpy()
    n = len(coords)
    lists = oracle.build_map(coords, 3).lists
    x = x.double().cpu().requires_grad_()
    conv = torch.zeros(n, e.CHANNELS, dtype=torch.float64)
    for k in range(27):
        i, o = (torch.as_tensor(np.asarray(v), dtype=torch.long) for v in lists[k])
        conv = conv.index_add(0, o, x[i] @ w["conv"][k])
    h1 = x + conv
    qkv = (_norm(h1, w["norm1"]) @ w["qkv"] + w["qkv_bias"]).view(n, -1, e.DIM)
    parts = qkv.split([e.HEADS, e.KV_HEADS, e.KV_HEADS], 1)
    table = block.table.double().cpu()
    pos = torch.as_tensor(coords[:, 1:]).long()
    c, s = (torch.cat([table[pos[:, a], :, i] for a in range(3)], 1)[:, None] for i in (0, 1))
    turned = []
    for t, name in zip(parts[:2], ("q_norm", "k_norm")):
        a, b, rest = _norm(t, w[name]).split([6, 6, e.DIM - 12], -1)
        turned.append(torch.cat([a * c - b * s, a * s + b * c, rest], -1))
    q, k = turned
    made = []
    cu = block.windows.cpu().tolist()
    for lo, hi in zip(cu, cu[1:]):
        heads = []
        for h in range(e.HEADS):
            g = h // (e.HEADS // e.KV_HEADS)
            p = torch.softmax(q[lo:hi, h] @ k[lo:hi, g].T / math.sqrt(e.DIM), -1)
            heads.append(p @ parts[2][lo:hi, g])
        made.append(torch.stack(heads, 1))
    h2 = h1 + torch.cat(made).reshape(n, -1) @ w["proj"] + w["proj_bias"]
    y2 = _norm(h2, w["norm2"])
    out = []
    cu = block.bands.cpu().tolist()
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        z = y2[lo:hi] @ w["up"][b] + w["up_bias"][b]
        u = 0.5 * z * torch.erfc(-z / math.sqrt(2))
        out.append(h2[lo:hi] + u @ w["down"][b] + w["down_bias"][b])
    out = torch.cat(out)
    out.backward(grad.double().cpu())
    return out.detach(), x.grad, {n: t.grad for n, t in w.items()}


def _relative(got, ref):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape
    return float((got - ref).norm() / ref.norm())


def test_block_and_its_gradients(example):
    """bf16 stores about ten tensors on the way to the output and to each
    gradient, each off by at most 2^-8 of its values: 10 x 2^-8 of the norm."""
    coords = workloads.random_grid(seed=3, extent=40, occupancy=0.05, batches=2)
    block = example.Block(coords)
    sizes = np.diff(block.bands.cpu().numpy())
    assert len(sizes) == example.BANDS and sizes.sum() == len(coords)
    n = len(coords)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, example.CHANNELS, generator=g).cuda().bfloat16()
    grad = torch.randn(n, example.CHANNELS, generator=g).cuda().bfloat16()
    out, saved = block.forward(x)
    gx, grads = block.backward(grad, saved)
    ref, ref_gx, ref_grads = _reference(block, example, x, grad)
    assert set(grads) == set(ref_grads)
    bound = 10 * 2.0 ** -8
    assert _relative(out, ref) < bound
    assert _relative(gx, ref_gx) < bound
    for name, got in grads.items():
        assert _relative(got, ref_grads[name]) < bound, name


def test_training_runs(example):
    coords = workloads.random_grid(seed=4, extent=30, occupancy=0.05, batches=1)
    errors = example.train(coords, 3)
    assert len(errors) == 3 and all(math.isfinite(e) for e in errors)


def test_bands_without_voxels(example):
    """All voxels in one window: the other bands' weights get zero gradients."""
    coords = workloads.random_grid(seed=6, extent=12, occupancy=0.3, batches=1)
    block = example.Block(coords)
    x = torch.randn(len(coords), example.CHANNELS, device="cuda").bfloat16()
    out, saved = block.forward(x)
    _, grads = block.backward(out, saved)
    empty = [b for b, size in enumerate(np.diff(block.bands.cpu().numpy())) if size == 0]
    assert empty
    for name in ("up", "up_bias", "down", "down_bias"):
        assert not bool(grads[name][empty].any()) and bool(grads[name].isfinite().all())
