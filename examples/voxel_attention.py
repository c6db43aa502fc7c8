"""A transformer block over voxels: sparse convolution, head norm with the
voxel coordinates rotated in, attention among the voxels of each window, and a
training step through all of it.

    python examples/voxel_attention.py [--steps N]

The rows of a batch of frames are sorted by window (16 x 16 x 16 voxels), so
that a window's voxels are one packed sequence.  The block computes

    x  = x + conv3(x)                              (submanifold, 3 x 3 x 3)
    q, k, v = conv1(x)                             (K = 1: a projection)
    q, k = norm_rotary(q, k, coordinates)
    x  = x + conv1(attention(q, k, v, windows))

with grouped heads (8 queries, 2 keys), and its backward pass calls the
gradient of each operator in turn; the weights take a plain gradient step.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import submanifold_sparse_convolution_device_amd as sp  # noqa: E402
import workloads  # noqa: E402

CHANNELS, HEADS, KV_HEADS, DIM, WINDOW = 128, 8, 2, 16, 16
QKV = (HEADS + 2 * KV_HEADS) * DIM


def windows(coords):
    """The row order that packs each window, and the windows' row offsets."""
    key = np.concatenate([coords[:, :1], coords[:, 1:] // WINDOW], 1)
    _, number = np.unique(key, axis=0, return_inverse=True)
    order = np.argsort(number.reshape(-1), kind="stable")
    counts = np.bincount(number.reshape(-1))
    return order, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


class Block:
    """The block's weights (fp32 masters, bf16 copies for the products) and
    its forward and backward passes over one batch of frames."""

    def __init__(self, coords, device="cuda"):
        order, cu = windows(coords)
        self.coords = torch.from_numpy(np.ascontiguousarray(coords[order])).to(device)
        self.cu = torch.from_numpy(cu).to(device)
        self.map3, self.map1 = sp.build_map(self.coords, 3), sp.build_map(self.coords, 1)
        extent = int(coords[:, 1:].max()) + 1
        self.table = sp.rotary_table(extent, 2, base=100.0, device=device)  # 12 of a head's 16 elements turn
        g = torch.Generator().manual_seed(0)

        def draw(*shape, fan):
            return (torch.randn(*shape, generator=g) / fan ** 0.5).to(device)

        self.weights = {
            "conv": draw(27, CHANNELS, CHANNELS, fan=27 * CHANNELS),
            "qkv": draw(1, CHANNELS, QKV, fan=CHANNELS),
            "out": draw(1, HEADS * DIM, CHANNELS, fan=HEADS * DIM),
            "q_norm": torch.ones(DIM, device=device),
            "k_norm": torch.ones(DIM, device=device),
        }

    def forward(self, x):
        w = {n: t.bfloat16() for n, t in self.weights.items()}
        n = x.shape[0]
        x1 = x + sp.forward(x, w["conv"], self.map3)
        qkv = sp.forward(x1, w["qkv"], self.map1).view(n, -1, DIM)
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        qr, kr = sp.norm_rotary(q, k, w["q_norm"], w["k_norm"], self.table, self.coords[:, 1:])
        a, lse = sp.attention(qr, kr, v, self.cu, return_lse=True)
        y = x1 + sp.forward(a.view(n, -1), w["out"], self.map1)
        return y, (w, x, x1, q, k, v, qr, kr, a, lse)

    def backward(self, grad, saved):
        w, x, x1, q, k, v, qr, kr, a, lse = saved
        n = x.shape[0]
        grads = {"out": sp.backward_weights(a.view(n, -1), grad, self.map1)}
        ga = sp.backward_data(grad, w["out"], self.map1).view(n, HEADS, DIM)
        gqkv = torch.empty(n, HEADS + 2 * KV_HEADS, DIM, dtype=x.dtype, device=x.device)
        gq, gk, gv = gqkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        sp.attention_backward(ga, qr, kr, v, a, lse, self.cu, grads=(gq, gk, gv))
        _, _, grads["q_norm"], grads["k_norm"] = sp.norm_rotary_backward(
            gq, gk, q, k, w["q_norm"], w["k_norm"], self.table, self.coords[:, 1:], grads=(gq, gk))
        gqkv = gqkv.view(n, QKV)
        grads["qkv"] = sp.backward_weights(x1, gqkv, self.map1)
        g1 = grad + sp.backward_data(gqkv, w["qkv"], self.map1)
        grads["conv"] = sp.backward_weights(x, g1, self.map3)
        return g1 + sp.backward_data(g1, w["conv"], self.map3), grads


def train(coords, steps, rate=0.5, seed=1):
    """Fits the block's output to fixed targets; returns the mean squared
    errors before each step."""
    block = Block(coords)
    n = block.coords.shape[0]
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, CHANNELS, generator=g).cuda().bfloat16()
    target = torch.randn(n, CHANNELS, generator=g).cuda()
    errors = []
    for _ in range(steps):
        y, saved = block.forward(x)
        diff = y.float() - target
        errors.append(float(diff.square().mean()))
        _, grads = block.backward((2 * diff / CHANNELS).bfloat16(), saved)
        for name, grad in grads.items():
            block.weights[name] -= rate / n * grad
    return errors


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=10)
    steps = ap.parse_args().steps
    coords = workloads.lidar_frame(seed=1)
    print(f"{coords.shape[0]} voxels in {len(windows(coords)[1]) - 1} windows")
    for i, e in enumerate(train(coords, steps)):
        print(f"step {i}: mean squared error {e:.4f}")


if __name__ == "__main__":
    main()
