"""The transformer block of examples/voxel_attention.py: its gradients against
the same block in 64-bit torch with autograd, and a few training steps."""
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
    import voxel_attention
    return voxel_attention


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
    x1 = x + conv
    qkv = (x1 @ w["qkv"][0]).view(n, -1, e.DIM)
    parts = qkv.split([e.HEADS, e.KV_HEADS, e.KV_HEADS], 1)
    table = block.table.double().cpu()
    pos = torch.as_tensor(coords[:, 1:]).long()
    c, s = (torch.cat([table[pos[:, a], :, i] for a in range(3)], 1)[:, None] for i in (0, 1))
    turned = []
    for t, name in zip(parts[:2], ("q_norm", "k_norm")):
        y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w[name]
        a, b, rest = y[..., :6], y[..., 6:12], y[..., 12:]
        turned.append(torch.cat([a * c - b * s, a * s + b * c, rest], -1))
    q, k = turned
    out = []
    cu = block.cu.cpu().tolist()
    for lo, hi in zip(cu, cu[1:]):
        heads = []
        for h in range(e.HEADS):
            g = h // (e.HEADS // e.KV_HEADS)
            p = torch.softmax(q[lo:hi, h] @ k[lo:hi, g].T / math.sqrt(e.DIM), -1)
            heads.append(p @ parts[2][lo:hi, g])
        out.append(torch.stack(heads, 1))
    y = x1 + torch.cat(out).reshape(n, -1) @ w["out"][0]
    y.backward(grad.double().cpu())
    return y.detach(), x.grad, {name: t.grad for name, t in w.items()}


def test_block_against_autograd(example):
    """bf16 rounds every intermediate once (2^-9 of it, in the root mean
    square): over the block's eight stages the relative error stays within
    8 x 2^-8."""
    coords = workloads.random_grid(seed=3, extent=20, occupancy=0.05, batches=2)
    block = example.Block(coords)
    n = block.coords.shape[0]
    g = torch.Generator().manual_seed(2)
    x = torch.randn(n, example.CHANNELS, generator=g).bfloat16().cuda()
    grad = torch.randn(n, example.CHANNELS, generator=g).bfloat16().cuda()
    y, saved = block.forward(x)
    gx, grads = block.backward(grad, saved)
    want_y, want_gx, want = _reference(block, example, x, grad)

    def off(a, b):
        return float((a.double().cpu().reshape(b.shape) - b).norm() / b.norm())

    assert off(y, want_y) <= 8 * 2.0 ** -8
    assert off(gx, want_gx) <= 8 * 2.0 ** -8
    for name in grads:
        assert off(grads[name], want[name]) <= 8 * 2.0 ** -8, name


def test_training_lowers_the_error(example):
    errors = example.train(workloads.random_grid(seed=4, extent=24, occupancy=0.04, batches=2), steps=8)
    assert all(math.isfinite(e) for e in errors)
    assert errors[-1] < 0.97 * errors[0]
