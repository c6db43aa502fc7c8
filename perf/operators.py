"""The transformer operators over packed voxel rows, as they are measured.

A point-cloud transformer block runs, next to the sparse convolutions:

- ``norm_rotary``: the RMS norm of every head of the queries and keys with the
  position rotation (one position axis, or the three voxel coordinates) in the
  same pass, and its gradient (with the gradients of the two norm weights);
- ``attention``: softmax attention over packed sequences of different lengths
  (a frame's or a window's voxels), with grouped heads, causal or inside a
  band, also for single queries over long keys, and its gradient.

A case's ``op`` is one of the two, ``train`` adds the gradients to the pass.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases


def _attention(name, train, dtype, heads, kv_heads, dim, batch, low, high, queries=0, causal=False, left=-1,
               layout=1):
    """``batch`` sequences of low..high rows each; queries > 0: that many
    queries at the end of every sequence instead of all of its rows."""
    return {"name": name, "op": "attention", "train": train, "dtype": dtype, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "batch": batch, "low": low, "high": high, "queries": queries, "causal": causal, "left": left,
            "layout": layout}


def _norm_rotary(name, train, dtype, rows, heads, kv_heads, dim, rotary, axes, interleaved):
    return {"name": name, "op": "norm_rotary", "train": train, "dtype": dtype, "rows": rows, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rotary": rotary, "axes": axes, "interleaved": interleaved}


def listed():
    return [
        # a handful of voxel windows of one small object: the call's latency
        _attention("attend_windows_small", False, "bf16", 4, 4, 16, 64, 0, 64),
        # whole frames at a coarse level of a stack, 256 channels in 8 heads
        _attention("attend_frames", False, "f16", 8, 8, 32, 8, 500, 4000),
        # long ordered sequences, grouped heads
        _attention("attend_causal_long", False, "bf16", 16, 4, 128, 4, 1000, 8192, causal=True),
        # one new query for each of many long sequences, as when voxels are generated one by one
        _attention("attend_single_query", False, "bf16", 16, 2, 128, 24, 1, 24000, queries=1, causal=True),
        # rows in scan order that look back over a fixed number of rows, fp32, an odd head size
        _attention("attend_band_f32", False, "f32", 6, 3, 40, 5, 100, 2500, causal=True, left=200),
        # training over the windows (up to 7 x 7 x 7 voxels) of a batch of frames, 256 channels
        _attention("train_windows", True, "bf16", 8, 8, 32, 1200, 0, 343),
        # training over ordered sequences, grouped heads
        _attention("train_causal", True, "f16", 8, 2, 64, 6, 200, 4096, causal=True),
        # training over whole frames in fp32, few channels
        _attention("train_frames_f32", True, "f32", 2, 2, 24, 3, 700, 1500),
        # the voxels of one small object: the call's latency
        _norm_rotary("rotate_object", False, "f16", 700, 4, 4, 16, 12, 3, False),
        # 8 frames' voxels, 256 channels in 8 heads, rotated by their coordinates
        _norm_rotary("rotate_frames", False, "bf16", 800000, 8, 8, 32, 24, 3, True),
        # training over ordered sequences, grouped heads, half of each head rotated
        _norm_rotary("train_rotate_ordered", True, "bf16", 120001, 16, 4, 128, 64, 1, False),
        # training in fp32, an odd head size
        _norm_rotary("train_rotate_f32", True, "f32", 30011, 6, 3, 40, 36, 3, True),
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    train = rng.random() < 0.5
    if rng.random() < 0.4:
        dim = rng.choice([16, 24, 32, 40, 48, 64, 80, 96, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        axes = rng.choice([1, 3])
        rotary = dim - dim % (2 * axes) if rng.random() < 0.6 else 2 * axes * max(1, dim // (4 * axes))
        most = 800000 * 16 * 32 // ((heads + kv_heads) * dim * SIZES[dtype] // 2) // (3 if train else 1)
        case = _norm_rotary("", train, dtype, _spread(rng, 1, most), heads, kv_heads, dim, rotary, axes,
                            rng.random() < 0.5)
    else:
        dim = rng.choice([16, 24, 32, 40, 48, 64, 80, 96, 128])
        kv_heads = rng.choice([1, 2, 3, 4])
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        causal = rng.random() < 0.6
        left = _spread(rng, 16, 1000) if causal and rng.random() < 0.3 else -1
        if not train and rng.random() < 0.3:
            queries = rng.choice([1, 1, 1, 2, 5])
            high = _spread(rng, 32, 24000)
            batch = _spread(rng, 1, min(200, max(1, 24 * 24000 // high)))
        else:
            queries = 0
            high = _spread(rng, 16, 2500 if dtype == "f32" else 6000)
            budget = (0.3 if dtype == "f32" or train else 1.0) * 16 * 8192.0 ** 2
            batch = _spread(rng, 1, max(1, min(1000, int(budget / (heads * float(high) ** 2)))))
        case = _attention("", train, dtype, heads, kv_heads, dim, batch, rng.choice([0, 1, high // 8, high // 2]), high,
                          queries, causal, left, rng.randrange(1 << 20))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """Rows of each sequence: the case's own, so that its work is known."""
    rng = random.Random(case["layout"])
    got = [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    got[rng.randrange(len(got))] = case["high"]
    return got


def _query_lengths(case):
    return [case["queries"]] * case["batch"] if case["queries"] else _lengths(case)


def _offsets(lengths, device):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=device)


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=device) * scale).to(dt)

    s = {"case": case}
    if case["op"] == "attention":
        lengths, q_lengths = _lengths(case), _query_lengths(case)
        rows, q_rows = sum(lengths), sum(q_lengths)
        s["cu_k"] = _offsets(lengths, device)
        s["longest_k"], s["longest_q"] = max(lengths), max(q_lengths)
        if case["queries"]:
            s["cu_q"] = _offsets(q_lengths, device)
            s["q"] = normal(q_rows, h, d)
            kv = normal(rows, 2 * hk, d)
            s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
        else:  # one projection's output holds all three
            s["cu_q"] = s["cu_k"]
            qkv = normal(rows, h + 2 * hk, d)
            s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if case["train"]:
            s["grad"] = normal(q_rows, h, d)
        return s
    n, axes, rotary = case["rows"], case["axes"], case["rotary"]
    qkv = normal(n, h + 2 * hk, d, scale=1.7)
    s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + hk]
    s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=device)).to(dt)
    s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=device)).to(dt)
    extent = 8192 if axes == 1 else 2048
    if axes == 1:  # a row's place in its sequence
        s["positions"] = (torch.arange(n, device=device) % extent).to(torch.int32).view(n, 1)
    else:  # the voxel coordinates (b, z, y, x), as the maps take them
        coords = torch.randint(0, extent, (n, 4), generator=g, device=device, dtype=torch.int32)
        coords[:, 1] %= 256
        s["positions"] = coords[:, 1:]
    pairs = rotary // (2 * axes)
    base = 10000.0 if axes == 1 else 100.0
    angle = (torch.arange(extent, dtype=torch.float64, device=device)[:, None]
             * base ** (-torch.arange(pairs, dtype=torch.float64, device=device) / pairs))
    s["table"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    if case["train"]:
        s["grad_q"], s["grad_k"] = normal(n, h, d), normal(n, hk, d)
    return s


# ------------------------------------------------------------------ a pass


def run(s):
    case = s["case"]
    if case["op"] == "attention":
        return _own_attention(s, case) if own else _plain_attention(s, case)
    return _own_norm_rotary(s, case) if own else _plain_norm_rotary(s, case)


def _own_attention(s, case):
    import submanifold_sparse_convolution_device_amd as sp
    how = {"causal": case["causal"], "window": (case["left"], -1)}
    out, lse = sp.attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], return_lse=True, **how)
    if not case["train"]:
        return {"out": out, "lse": lse}
    gq, gk, gv = sp.attention_backward(s["grad"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"], **how)
    return {"out": out, "lse": lse, "grad_q": gq, "grad_k": gk, "grad_v": gv}


def _own_norm_rotary(s, case):
    import submanifold_sparse_convolution_device_amd as sp
    how = {"rotary_dim": case["rotary"], "interleaved": case["interleaved"], "eps": 1e-6}
    rest = (s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"])
    q, k = sp.norm_rotary(*rest, **how)
    if not case["train"]:
        return {"q": q, "k": k}
    gq, gk, gqw, gkw = sp.norm_rotary_backward(s["grad_q"], s["grad_k"], *rest, **how)
    return {"q": q, "k": k, "grad_q": gq, "grad_k": gk, "grad_q_weight": gqw, "grad_k_weight": gkw}


def _pad(x, cu, longest):
    """[rows, heads, dim] -> fp32 [sequences, heads, longest, dim]; rows past a sequence's end are zero."""
    at = cu[:-1, None].long() + torch.arange(longest, device=x.device)
    there = at < cu[1:, None]
    rows = x[at.clamp(max=x.shape[0] - 1)].float() * there[..., None, None]
    return rows.transpose(1, 2).contiguous()


def _unpad(x, cu, total):
    """The inverse of _pad."""
    row = torch.arange(total, device=x.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    return x[b, :, row - cu[b]]


def _plain_attention(s, case):
    cu_q, cu_k = s["cu_q"], s["cu_k"]
    dt = s["q"].dtype
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = h // hk
    nq, nk = s["longest_q"], s["longest_k"]
    batch = cu_k.shape[0] - 1
    scale = d ** -0.5
    # the heads of a group follow one another along the rows of their shared key head
    q = _pad(s["q"], cu_q, nq).view(batch, hk, group * nq, d)
    k = _pad(s["k"], cu_k, nk)
    v = _pad(s["v"], cu_k, nk)
    len_q, len_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i = torch.arange(nq, device=q.device)[None, :, None]
    j = torch.arange(nk, device=q.device)[None, None, :]
    at = i + (len_k - len_q)[:, None, None]  # the key at which a query stands: the last ones meet
    seen = (i < len_q[:, None, None]) & (j < len_k[:, None, None])
    if case["causal"]:
        seen = seen & (j <= at)
    if case["left"] >= 0:
        seen = seen & (j >= at - case["left"])
    seen = seen[:, None, None].expand(batch, 1, group, nq, nk).reshape(batch, 1, group * nq, nk)
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p = p.div_(total.masked_fill(total == 0, 1.0))
    out = torch.matmul(p, v)
    rows = s["q"].shape[0]

    def back(x, cu, heads, n, total_rows):
        return _unpad(x.view(batch, heads, n, -1), cu, total_rows)

    got = {"out": back(out, cu_q, h, nq, rows).to(dt), "lse": back(lse, cu_q, h, nq, rows).squeeze(-1)}
    if case["train"]:
        grad = _pad(s["grad"], cu_q, nq).view(batch, hk, group * nq, d)
        grad_v = torch.matmul(p.transpose(-1, -2).contiguous(), grad)
        delta = (grad * out).sum(-1, keepdim=True)
        ds = torch.matmul(grad, v.transpose(-1, -2).contiguous()).sub_(delta).mul_(p).mul_(scale)
        grad_q = torch.matmul(ds, k)
        grad_k = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
        got["grad_q"] = back(grad_q, cu_q, h, nq, rows).to(dt)
        got["grad_k"] = back(grad_k, cu_k, hk, nk, s["k"].shape[0]).to(dt)
        got["grad_v"] = back(grad_v, cu_k, hk, nk, s["k"].shape[0]).to(dt)
    return got


def _split(x, rotary, interleaved):
    """The two members of every rotated pair, and what is not rotated."""
    if interleaved:
        return x[..., 0:rotary:2], x[..., 1:rotary:2], x[..., rotary:]
    return x[..., :rotary // 2], x[..., rotary // 2:rotary], x[..., rotary:]


def _join(a, b, rest, interleaved):
    pair = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([pair, rest], -1)


def _plain_norm_rotary(s, case):
    rotary, inter, d, dt = case["rotary"], case["interleaved"], case["dim"], s["q"].dtype
    angles = s["table"][s["positions"].long()]  # [rows, axes, pairs, 2]
    c = angles[..., 0].flatten(1)[:, None]
    sn = angles[..., 1].flatten(1)[:, None]
    got = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_weight"].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        a, b, rest = _split(x * r * w, rotary, inter)
        got[name] = _join(a * c - b * sn, a * sn + b * c, rest, inter).to(dt)
        if case["train"]:
            a, b, rest = _split(s["grad_" + name].float(), rotary, inter)
            g = _join(a * c + b * sn, b * c - a * sn, rest, inter)
            got["grad_" + name + "_weight"] = (g * x * r).sum((0, 1))
            g = g * w
            got["grad_" + name] = (r * (g - x * r * r * (g * x).mean(-1, keepdim=True))).to(dt)
    return got


# ------------------------------------------------------------------ work


def _visible(case):
    """Pairs of a query and a key that it sees, over all sequences of one head."""
    total = 0
    for nq, nk in zip(_query_lengths(case), _lengths(case)):
        at = np.arange(nq, dtype=np.int64) + (nk - nq)
        hi = np.minimum(at, nk - 1) if case["causal"] else np.full(nq, nk - 1, np.int64)
        lo = np.maximum(at - case["left"], 0) if case["left"] >= 0 else np.zeros(nq, np.int64)
        total += int(np.maximum(hi - lo + 1, 0).sum())
    return total


def work(case):
    h, hk, d, size = case["heads"], case["kv_heads"], case["dim"], SIZES[case["dtype"]]
    if case["op"] == "attention":
        rows, q_rows = sum(_lengths(case)), sum(_query_lengths(case))
        if case["queries"] and case["left"] >= 0:  # the keys that a band around the last rows reaches
            rows = sum(min(n, case["left"] + case["queries"]) for n in _lengths(case))
        qo, kv, lse = q_rows * h * d * size, rows * hk * d * size, q_rows * h * 4
        pairs = float(_visible(case)) * h
        if not case["train"]:
            return {"bytes": 2 * qo + 2 * kv + lse, "flops": 4 * pairs * d}
        # reads q, k, v and the output's gradient, writes the output and three gradients; two products
        # forward and five backward (the scores again, and four gradients')
        return {"bytes": 4 * qo + 4 * kv + lse, "flops": 14 * pairs * d}
    n, axes, rotary = case["rows"], case["axes"], case["rotary"]
    x = n * (h + hk) * d * size
    side = n * axes * 4 + 2 * d * size
    if not case["train"]:
        return {"bytes": 2 * x + side, "flops": n * (h + hk) * (4 * d + 3 * rotary)}
    return {"bytes": 4 * x + side + 2 * d * 4, "flops": n * (h + hk) * (14 * d + 6 * rotary)}


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(s, case) if case["op"] == "attention" else _exact_norm_rotary(s, case)


def _exact_attention(s, case):
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = h // hk
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    grads = [torch.zeros_like(x) for x in (q, k, v)] if case["train"] else None
    q0 = k0 = 0
    for nq, nk in zip(_query_lengths(case), _lengths(case)):
        if nq and nk:
            # a query at row i of nq stands at key i + nk - nq
            delta = torch.arange(nk, device=q.device)[None] - torch.arange(nk - nq, nk, device=q.device)[:, None]
            hidden = torch.zeros_like(delta, dtype=torch.bool)
            if case["causal"]:
                hidden |= delta > 0
            if case["left"] >= 0:
                hidden |= delta < -case["left"]
            blank = hidden.all(1)
            step = max(1, int(3e8 / (float(nq) * nk)))  # heads at a time
            for at in range(0, h, step):
                hs = torch.arange(at, min(h, at + step), device=q.device)
                ks = hs // group
                qs, kk, vv = q[q0:q0 + nq, hs], k[k0:k0 + nk, ks], v[k0:k0 + nk, ks]
                if grads is not None:
                    qs, kk, vv = (x.clone().requires_grad_() for x in (qs, kk, vv))
                logits = torch.einsum("ihd,jhd->hij", qs, kk) / math.sqrt(d)
                logits = torch.where(hidden, -math.inf, logits)
                norm = torch.logsumexp(torch.where(blank[:, None], 0.0, logits), -1, keepdim=True)
                p = torch.exp(logits - norm)
                o = torch.einsum("hij,jhd->ihd", p, vv)
                out[q0:q0 + nq, hs] = o.detach()
                row = torch.where(blank, -math.inf, norm.detach().squeeze(-1))
                lse[q0:q0 + nq, hs] = row.transpose(0, 1)
                if grads is not None:
                    got = torch.autograd.grad(o, (qs, kk, vv), s["grad"][q0:q0 + nq, hs].double())
                    grads[0][q0:q0 + nq, hs] = got[0]
                    grads[1][k0:k0 + nk].index_add_(1, ks, got[1])
                    grads[2][k0:k0 + nk].index_add_(1, ks, got[2])
        q0, k0 = q0 + nq, k0 + nk
    if grads is None:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "grad_q": grads[0], "grad_k": grads[1], "grad_v": grads[2]}


def _exact_norm_rotary(s, case):
    rotary, axes = case["rotary"], case["axes"]
    half, pairs = rotary // 2, rotary // (2 * axes)
    turn = torch.view_as_complex(s["table"].double())
    at = torch.arange(half, device=turn.device)
    turn = turn[s["positions"].long()[:, at // pairs], at % pairs][:, None]  # [rows, 1, pairs of all axes]
    if case["interleaved"]:
        first, second = 2 * at, 2 * at + 1
    else:
        first, second = at, at + half
    got = {}
    for name in ("q", "k"):
        x = s[name].double().requires_grad_(case["train"])
        w = s[name + "_weight"].double().requires_grad_(case["train"])
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        z = torch.complex(y[..., first], y[..., second]) * turn
        full = y.clone()
        full[..., first] = z.real
        full[..., second] = z.imag
        got[name] = full.detach()
        if case["train"]:
            gx, gw = torch.autograd.grad(full, (x, w), s["grad_" + name].double())
            got["grad_" + name], got["grad_" + name + "_weight"] = gx, gw
    return got
