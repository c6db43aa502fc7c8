"""The products and norms of a transformer block over packed voxel rows, as
they are measured.

Between the attention of such a block and the next one stand

- ``add_norm``: the residual's addition with the RMS norm of the whole row,
  and its gradient.  The sum is stored in the rows' type and the norm is of
  the stored sum;
- ``linear``: the matrix product with bias, activation and residual, and its
  gradients (fp32 for weights and bias).  Its input may be the activation of
  an earlier product (``before``): the gradient then goes on to that product's
  stored result;
- ``experts``: the same with weights of its own for each group of rows.  The
  groups are packed one after another, have any lengths and may be empty;
  rows behind the last one (a padded batch) give zeros.

A case's ``op`` is one of the three, ``train`` adds the gradients to the pass.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases


def _add_norm(name, train, dtype, rows, channels, residual=True):
    return {"name": name, "op": "add_norm", "train": train, "dtype": dtype, "rows": rows, "channels": channels,
            "residual": residual}


def _linear(name, train, dtype, rows, c_in, c_out, act="", residual=False, before=""):
    return {"name": name, "op": "linear", "train": train, "dtype": dtype, "rows": rows, "c_in": c_in, "c_out": c_out,
            "act": act, "residual": residual, "before": before}


def _experts(name, train, dtype, rows, groups, c_in, c_out, act="", before="", padding=0, layout=1):
    """``rows`` in all, the last ``padding`` of them in no group."""
    return {"name": name, "op": "experts", "train": train, "dtype": dtype, "rows": rows, "groups": groups,
            "c_in": c_in, "c_out": c_out, "act": act, "residual": False, "before": before, "padding": padding,
            "layout": layout}


def listed():
    return [
        # the voxels of one small object: the call's latency
        _add_norm("norm_object", False, "f16", 700, 128),
        # 8 frames' voxels, 256 channels
        _add_norm("norm_frames", False, "bf16", 800000, 256),
        # training at a model width of language models, an odd number of rows
        _add_norm("train_norm_wide", True, "bf16", 24001, 4096),
        # training in fp32 at a network's 96-channel level
        _add_norm("train_norm_f32", True, "f32", 100003, 96),
        # one new token for each of a few sequences: the weights' bytes
        _linear("linear_tokens", False, "bf16", 5, 2048, 8192, act="silu"),
        # the feed-forward's first product over the voxels of 4 frames
        _linear("linear_frames", False, "bf16", 400000, 256, 1024, act="gelu"),
        # the classes' scores of a frame in fp32: 20 columns
        _linear("linear_classes_f32", False, "f32", 120001, 96, 20),
        # training the feed-forward's second product: its input is the first one's activation
        _linear("train_feedforward", True, "bf16", 65537, 1024, 256, residual=True, before="gelu"),
        # training at a model width of language models
        _linear("train_linear_wide", True, "f16", 8192, 4096, 4096),
        # a few rows spread over many experts, most of them empty: the call's latency
        _experts("experts_tokens", False, "bf16", 64, 32, 512, 1024, act="relu", layout=3),
        # the voxels of 2 frames over experts of uneven share, in a padded batch
        _experts("experts_frames", False, "f16", 200000, 8, 256, 512, act="gelu", padding=1234, layout=5),
        # training experts in fp32
        _experts("train_experts_f32", True, "f32", 20011, 5, 128, 192, act="silu", layout=7),
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    train = rng.random() < 0.5
    size = SIZES[dtype]
    op = rng.choice(["add_norm", "linear", "linear", "experts"])
    if op == "add_norm":
        channels = 8 * _spread(rng, 2, 1024)
        most = 1600000000 // ((7 if train else 4) * channels * size)
        case = _add_norm("", train, dtype, _spread(rng, 1, most), channels, rng.random() < 0.8)
    else:
        if rng.random() < 0.7:
            c_in, c_out = (8 * _spread(rng, 2, 512) for _ in range(2))
        else:
            c_in, c_out = (_spread(rng, 3, 1000) for _ in range(2))
        by_bytes = 1500000000 / (size * (c_in + 2 * c_out) * (3 if train else 1))
        by_flops = (1e11 if dtype == "f32" else 8e11) / (2.0 * c_in * c_out * (3 if train else 1))
        most = max(1, int(min(by_bytes, by_flops)))
        rows = _spread(rng, 1, most)
        # the activation's gradient follows the stored product, which 16 bits round: in training it is fp32's
        act = rng.choice(["", "relu", "silu", "gelu"]) if dtype == "f32" or not train else ""
        before = rng.choice(["", "silu", "gelu"]) if train else ""
        if op == "linear":
            case = _linear("", train, dtype, rows, c_in, c_out, act, rng.random() < 0.4, before)
        else:
            groups = _spread(rng, 2, max(2, min(64, 30000000 // (c_in * c_out))))
            padding = rng.randint(0, rows // 8) if rng.random() < 0.3 else 0
            case = _experts("", train, dtype, rows, groups, c_in, c_out, act, before, padding, rng.randrange(1 << 20))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """Rows of each group: the case's own, so that its work is known.  Shares are uneven, some groups empty."""
    rng = random.Random(case["layout"])
    share = [0.0 if rng.random() < 0.15 else rng.random() ** 2 + 0.02 for _ in range(case["groups"])]
    if not any(share):
        share[rng.randrange(len(share))] = 1.0
    rows = case["rows"] - case["padding"]
    ends = [int(round(rows * c / sum(share))) for c in np.cumsum(share)]
    ends[-1] = rows
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=g, device=device) * scale + shift).to(dt)

    s = {"case": case}
    n = case["rows"]
    if case["op"] == "add_norm":
        c = case["channels"]
        s["x"] = normal(n, c)
        s["residual"] = normal(n, c, scale=2.0) if case["residual"] else None
        s["weight"] = normal(c, scale=0.2, shift=1.0)
        if case["train"]:
            s["grad_h"], s["grad_y"] = normal(n, c), normal(n, c)
        return s
    c_in, c_out = case["c_in"], case["c_out"]
    if case["before"]:  # as the product before stored them
        s["before"] = normal(n, c_in)
        s["x"] = _activation(case["before"], s["before"].float()).to(dt)
    else:
        s["x"] = normal(n, c_in)
    lead = ()
    if case["op"] == "experts":
        lead = (case["groups"],)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(_lengths(case))]), dtype=torch.int32, device=device)
    s["weight"] = normal(*lead, c_in, c_out, scale=c_in ** -0.5)
    s["bias"] = normal(*lead, c_out, scale=0.5)
    s["residual"] = normal(n, c_out) if case["residual"] else None
    if case["train"]:
        s["grad"] = normal(n, c_out)
    return s


# ------------------------------------------------------------------ a pass


def run(s):
    case = s["case"]
    if case["op"] == "add_norm":
        return _own_add_norm(s, case) if own else _plain_add_norm(s, case)
    return _own_linear(s, case) if own else _plain_linear(s, case)


def _own_add_norm(s, case):
    import submanifold_sparse_convolution_device_amd as sp
    h, y = sp.add_norm(s["x"], s["residual"], s["weight"], eps=EPS)
    if not case["train"]:
        return {"h": h, "y": y}
    grad, grad_weight = sp.add_norm_backward(s["grad_h"], s["grad_y"], h, s["weight"], eps=EPS)
    return {"h": h, "y": y, "grad": grad, "grad_weight": grad_weight}


def _own_linear(s, case):
    import submanifold_sparse_convolution_device_amd as sp
    cu = s.get("cu")
    keep = case["train"] and case["act"]
    out = sp.linear(s["x"], s["weight"], s["bias"], activation=case["act"] or None, residual=s["residual"], cu=cu,
                    return_pre=bool(keep))
    out, pre = out if keep else (out, None)
    got = {"out": out}
    if not case["train"]:
        return got
    grad = s["grad"]
    if keep:
        got["pre"] = pre
        got["grad_pre"] = grad = sp.activation_backward(grad, pre, case["act"])
    got["grad_x"], got["grad_weight"], got["grad_bias"] = sp.linear_backward(
        grad, s["x"], s["weight"], pre=s.get("before"), activation=case["before"] or None, cu=cu)
    return got


def _plain_add_norm(s, case):
    dt = s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    x, w = h.float(), s["weight"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    got = {"h": h, "y": (x * r * w).to(dt)}
    if case["train"]:
        g = s["grad_y"].float()
        got["grad_weight"] = (g * x * r).sum(0)
        t = g * w
        got["grad"] = (s["grad_h"].float() + r * (t - x * r * r * (t * x).mean(-1, keepdim=True))).to(dt)
    return got


def _activation(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 2 ** -0.5))
    return z


def _slope(name, z):
    """The activation's derivative."""
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        t = torch.sigmoid(z)
        return t * (1 + z * (1 - t))
    return 0.5 * (1 + torch.erf(z * 2 ** -0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _groups(case):
    """(group, first row, end) of the groups with rows; the whole batch is the only one of a dense product."""
    if case["op"] == "linear":
        return [(0, 0, case["rows"])]
    ends = np.cumsum(_lengths(case)).tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip([0] + ends[:-1], ends)) if b > a]


def _plain_linear(s, case):
    dt, act = s["x"].dtype, case["act"]
    x = s["x"].float()
    w, b = (t.float().reshape(-1, *t.shape[t.dim() - k:]) for t, k in ((s["weight"], 2), (s["bias"], 1)))
    groups = _groups(case)
    n, c_out = case["rows"], case["c_out"]
    pre = x.new_zeros(n, c_out) if case["op"] == "experts" else None
    for e, lo, hi in groups:
        z = torch.addmm(b[e], x[lo:hi], w[e])
        if pre is None:
            pre = z
        else:
            pre[lo:hi] = z
    out = _activation(act, pre)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    got = {"out": out.to(dt)}
    if not case["train"]:
        return got
    grad = s["grad"]
    if act:
        got["pre"] = pre.to(dt)
        got["grad_pre"] = grad = (grad.float() * _slope(act, got["pre"].float())).to(dt)
    grad = grad.float()
    gx, gw, gb = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
    for e, lo, hi in groups:
        torch.matmul(grad[lo:hi], w[e].t(), out=gx[lo:hi])
        torch.matmul(x[lo:hi].t(), grad[lo:hi], out=gw[e])
        torch.sum(grad[lo:hi], 0, out=gb[e])
    if case["before"]:
        gx = gx * _slope(case["before"], s["before"].float())
    got["grad_x"] = gx.to(dt)
    got["grad_weight"], got["grad_bias"] = gw.view(s["weight"].shape), gb.view(s["bias"].shape)
    return got


# ------------------------------------------------------------------ work


def work(case):
    n, size = case["rows"], SIZES[case["dtype"]]
    if case["op"] == "add_norm":
        c, res = case["channels"], case["residual"]
        row = n * c * size
        if not case["train"]:
            return {"bytes": row * (4 if res else 2) + c * size, "flops": 5 * n * c}
        # reads x, the residual and two gradients, writes the sum, the norm and a gradient
        return {"bytes": row * (7 if res else 5) + c * (size + 4), "flops": 15 * n * c}
    c_in, c_out = case["c_in"], case["c_out"]
    groups = _groups(case)
    used, there = len(groups), sum(b - a for _, a, b in groups)
    weights = used * (c_in + 1) * c_out
    macs = float(there) * c_in * c_out
    moved = there * c_in * size + weights * size + n * c_out * size * (2 if case["residual"] else 1)
    if not case["train"]:
        return {"bytes": moved, "flops": 2 * macs}
    # reads the gradient (and x's stored product), writes x's gradient and the weights'
    moved += there * c_out * size + n * c_in * size + case.get("groups", 1) * (c_in + 1) * c_out * 4
    if case["act"]:
        moved += 2 * n * c_out * size
    if case["before"]:
        moved += there * c_in * size
    return {"bytes": moved, "flops": 6 * macs}


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_add_norm(s, case) if case["op"] == "add_norm" else _exact_linear(s, case)


def _exact_add_norm(s, case):
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
    stored = h.to(s["x"].dtype).double().requires_grad_(case["train"])  # the norm is of the stored sum
    w = s["weight"].double().requires_grad_(case["train"])
    y = stored / torch.sqrt((stored * stored).mean(-1, keepdim=True) + EPS) * w
    got = {"h": h, "y": y.detach()}
    if case["train"]:
        through, got["grad_weight"] = torch.autograd.grad(y, (stored, w), s["grad_y"].double())
        got["grad"] = through + s["grad_h"].double()
    return got


_EXACT = {
    "": lambda z: z,
    "relu": torch.nn.functional.relu,
    "silu": torch.nn.functional.silu,
    "gelu": torch.nn.functional.gelu,
}


def _exact_linear(s, case):
    dense = case["op"] == "linear"
    x = s["x"].double()
    w = s["weight"].double()
    b = s["bias"].double()
    if dense:
        w, b = w[None], b[None]
    n, c_out = case["rows"], case["c_out"]
    which = torch.full((n,), -1, dtype=torch.int64)  # a row's group
    if dense:
        which[:] = 0
    else:
        of = torch.repeat_interleave(torch.arange(case["groups"]), torch.tensor(_lengths(case)))
        which[:of.shape[0]] = of
    rows = [torch.nonzero(which == e)[:, 0].to(x.device) for e in range(w.shape[0])]
    pre = torch.zeros(n, c_out, dtype=torch.float64, device=x.device)
    for e, at in enumerate(rows):
        if at.numel():
            pre[at] = x[at] @ w[e] + b[e]
    out = _EXACT[case["act"]](pre)
    if s["residual"] is not None:
        out = out + s["residual"].double()
    got = {"out": out}
    if not case["train"]:
        return got
    grad = s["grad"].double()
    if case["act"]:
        got["pre"] = pre
        leaf = pre.clone().requires_grad_()
        got["grad_pre"], = torch.autograd.grad(_EXACT[case["act"]](leaf), leaf, grad)
        grad = got["grad_pre"]
    gx = torch.zeros_like(x)
    gw, gb = torch.zeros_like(w), torch.zeros_like(b)
    for e, at in enumerate(rows):
        if at.numel():
            g = grad[at]
            gx[at] = g @ w[e].transpose(0, 1).contiguous()
            gw[e] = x[at].transpose(0, 1).contiguous() @ g
            gb[e] = g.sum(0)
    if case["before"]:
        leaf = s["before"].double().requires_grad_()
        gx, = torch.autograd.grad(_EXACT[case["before"]](leaf), leaf, gx)
    got["grad_x"] = gx
    got["grad_weight"], got["grad_bias"] = (gw[0], gb[0]) if dense else (gw, gb)
    return got
