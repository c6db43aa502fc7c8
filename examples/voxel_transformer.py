"""A pre-norm transformer block over voxels with experts by range, and a
training step through all of it.

    python examples/voxel_transformer.py [--steps N]

The rows of a batch of frames are sorted by range band (near, middle, far) and
within it by window (16 x 16 x 16 voxels), so that a band's rows and a window's
voxels are both packed one after another.  The block computes

    h1, y1  = add_norm(x, conv3(x))                  (submanifold, 3 x 3 x 3)
    q, k, v = linear(y1);  q, k = norm_rotary(q, k, coordinates)
    h2, y2  = add_norm(h1, linear(attention(q, k, v, windows)))
    out     = h2 + linear(gelu(linear(y2)))          (each band has weights of its own)

and its backward pass calls the gradient of each operator in turn.  The
feed-forward's activation and its slope run inside its products, the last
addition inside the second one, and each of the others with a norm.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import submanifold_sparse_convolution_device_amd as sp  # noqa: E402
import workloads  # noqa: E402

CHANNELS, HEADS, KV_HEADS, DIM, WINDOW, WIDE, BANDS = 128, 8, 2, 16, 16, 512, 3
QKV = (HEADS + 2 * KV_HEADS) * DIM


def packing(coords):
    """The row order, and the row offsets of the windows and of the bands.  A
    window's band is that of its distance from the middle of the frame."""
    window = np.concatenate([coords[:, :1], coords[:, 1:] // WINDOW], 1)
    middle = (coords[:, 2:].max(0) + coords[:, 2:].min(0)) / (2 * WINDOW)
    reach = np.hypot(*(window[:, 2:] + 0.5 - middle).T)
    band = np.minimum(reach / (reach.max() + 1e-9) * BANDS, BANDS - 1).astype(np.int64)
    _, number = np.unique(np.concatenate([band[:, None], window], 1), axis=0, return_inverse=True)
    order = np.argsort(number.reshape(-1), kind="stable")
    offsets = [np.concatenate([[0], np.cumsum(np.bincount(k))]).astype(np.int32)
               for k in (number.reshape(-1), np.append(band, BANDS - 1))]
    offsets[1][-1] -= 1  # (a last band without voxels still has its offsets)
    return order, *offsets


class Block:
    """The block's weights (fp32 masters, bf16 copies for the products) and
    its forward and backward passes over one batch of frames."""

    def __init__(self, coords, device="cuda"):
        order, windows, bands = packing(coords)
        self.coords = torch.from_numpy(np.ascontiguousarray(coords[order])).to(device)
        self.windows, self.bands = (torch.from_numpy(c).to(device) for c in (windows, bands))
        self.map3 = sp.build_map(self.coords, 3)
        self.table = sp.rotary_table(int(coords[:, 1:].max()) + 1, 2, base=100.0, device=device)
        g = torch.Generator().manual_seed(0)

        def draw(*shape, fan):
            return (torch.randn(*shape, generator=g) / fan ** 0.5).to(device)

        self.weights = {
            "conv": draw(27, CHANNELS, CHANNELS, fan=27 * CHANNELS),
            "qkv": draw(CHANNELS, QKV, fan=CHANNELS), "qkv_bias": draw(QKV, fan=100),
            "proj": draw(HEADS * DIM, CHANNELS, fan=HEADS * DIM), "proj_bias": draw(CHANNELS, fan=100),
            "up": draw(BANDS, CHANNELS, WIDE, fan=CHANNELS), "up_bias": draw(BANDS, WIDE, fan=100),
            "down": draw(BANDS, WIDE, CHANNELS, fan=WIDE), "down_bias": draw(BANDS, CHANNELS, fan=100),
            "norm1": torch.ones(CHANNELS, device=device), "norm2": torch.ones(CHANNELS, device=device),
            "q_norm": torch.ones(DIM, device=device), "k_norm": torch.ones(DIM, device=device),
        }

    def forward(self, x):
        w = {n: t.bfloat16() for n, t in self.weights.items()}
        n = x.shape[0]
        h1, y1 = sp.add_norm(x, sp.forward(x, w["conv"], self.map3), w["norm1"])
        q, k, v = sp.linear(y1, w["qkv"], w["qkv_bias"]).view(n, -1, DIM).split([HEADS, KV_HEADS, KV_HEADS], 1)
        qr, kr = sp.norm_rotary(q, k, w["q_norm"], w["k_norm"], self.table, self.coords[:, 1:])
        a, lse = sp.attention(qr, kr, v, self.windows, return_lse=True)
        h2, y2 = sp.add_norm(h1, sp.linear(a.view(n, -1), w["proj"], w["proj_bias"]), w["norm2"])
        u, pre = sp.linear(y2, w["up"], w["up_bias"], activation="gelu", cu=self.bands, return_pre=True)
        out = sp.linear(u, w["down"], w["down_bias"], residual=h2, cu=self.bands)
        return out, (w, x, h1, y1, q, k, v, qr, kr, a, lse, h2, y2, u, pre)

    def backward(self, grad, saved):
        w, x, h1, y1, q, k, v, qr, kr, a, lse, h2, y2, u, pre = saved
        n, g = x.shape[0], {}
        gpre, g["down"], g["down_bias"] = sp.linear_backward(grad, u, w["down"], pre=pre, activation="gelu", cu=self.bands)
        gy2, g["up"], g["up_bias"] = sp.linear_backward(gpre, y2, w["up"], cu=self.bands)
        gh2, g["norm2"] = sp.add_norm_backward(grad, gy2, h2, w["norm2"])
        ga, g["proj"], g["proj_bias"] = sp.linear_backward(gh2, a.view(n, -1), w["proj"])
        gqkv = torch.empty(n, HEADS + 2 * KV_HEADS, DIM, dtype=x.dtype, device=x.device)
        gq, gk, gv = gqkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        sp.attention_backward(ga.view(n, HEADS, DIM), qr, kr, v, a, lse, self.windows, grads=(gq, gk, gv))
        _, _, g["q_norm"], g["k_norm"] = sp.norm_rotary_backward(
            gq, gk, q, k, w["q_norm"], w["k_norm"], self.table, self.coords[:, 1:], grads=(gq, gk))
        gy1, g["qkv"], g["qkv_bias"] = sp.linear_backward(gqkv.view(n, QKV), y1, w["qkv"])
        gh1, g["norm1"] = sp.add_norm_backward(gh2, gy1, h1, w["norm1"])
        g["conv"] = sp.backward_weights(x, gh1, self.map3)
        return gh1 + sp.backward_data(gh1, w["conv"], self.map3), g


def train(coords, steps, rate=0.2, seed=1):
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
    _, windows, bands = packing(coords)
    print(f"{coords.shape[0]} voxels in {len(windows) - 1} windows, bands of {np.diff(bands).tolist()} rows")
    for i, e in enumerate(train(coords, steps)):
        print(f"step {i}: mean squared error {e:.4f}")


if __name__ == "__main__":
    main()
