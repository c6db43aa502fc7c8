"""Attention over packed sequences and the head norm with the position
rotation, in 64 bits on the CPU, with the rounding bounds the library's
kernels are held to.

Every bound is a first-order sum of roundings on the way from the inputs to
the value, each against the magnitudes that it acts on:

- u is the dtype's unit roundoff (2^-8, 2^-11, 2^-24), e = 2^-24 fp32's.
- A score is an fp32 sum of d products: d e times s_abs = scale sum |q||k|.
  exp(s - lse) adds the roundings of its argument (the constant, the
  difference and lse, at most 4 e times s_abs + log n), one ulp of exp2 (2 e)
  and, in lse, the sum of n terms (n e at most): relative
  eps = (2 d + 16) e max_j s_abs + (n + 16 + 8 log n) e.
- The 16-bit types round each probability and score gradient once as an
  operand (u relative; fp16 below its normal range 2^-25 absolute, of values
  scaled so that 2^8 is the largest).
- A sum of n terms in fp32, in any order: n e times the sum of magnitudes.
- The result's own rounding: u relative (fp16 below its normal range: 2^-25).
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E = 2.0 ** -24


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def offsets(lengths, start=0):
    cu = [start]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


def visible(nq, nk, causal, window):
    place = torch.arange(nq)[:, None] + nk - nq
    key = torch.arange(nk)[None]
    seen = torch.ones(nq, nk, dtype=torch.bool)
    left, right = window
    if causal:
        right = 0
    if left >= 0:
        seen &= key >= place - left
    if right >= 0:
        seen &= key <= place + right
    return seen


def attention(q, k, v, cu_q, cu_k, causal=False, window=(-1, -1), scale=None, grad=None):
    """A dict of out, lse (and grad_q, grad_k, grad_v), each with a bound
    under its name + "_tol"; rows of no sequence see no key."""
    dt, d = q.dtype, q.shape[2]
    u, group = U[dt], q.shape[1] // k.shape[1]
    # roundings of the operands of a second product
    up = u if dt != torch.float32 else 0.0
    scale = d ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    r = {"out": torch.zeros_like(q), "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64)}
    r["out_tol"], r["lse_tol"] = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64)
    if grad is not None:
        grad = grad.double()
        for n, x in (("grad_q", q), ("grad_k", k), ("grad_v", v)):
            r[n], r[n + "_tol"] = torch.zeros_like(x), torch.zeros_like(x)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        if q1 <= q0 or k1 <= k0:
            continue
        seen = visible(q1 - q0, k1 - k0, causal, window)
        n = k1 - k0
        for h in range(q.shape[1]):
            g = h // group
            Q, K, V = q[q0:q1, h], k[k0:k1, g], v[k0:k1, g]
            s = (Q @ K.T) * scale
            s_abs = (Q.abs() @ K.abs().T) * scale
            hidden = torch.where(seen, s, torch.tensor(-math.inf, dtype=torch.float64))
            lse = torch.logsumexp(hidden, -1)
            empty = ~seen.any(-1)
            P = torch.where(seen, torch.exp(s - torch.where(empty, 0.0, lse)[:, None]), 0.0)
            top = torch.where(seen, s_abs, 0.0).amax(-1, keepdim=True)
            eps = (2 * d + 16) * E * top + (n + 16 + 8 * math.log(n + 1)) * E
            O = P @ V
            r["out"][q0:q1, h] = O
            r["lse"][q0:q1, h] = lse
            r["lse_tol"][q0:q1, h] = torch.where(empty, 0.0, eps[:, 0] + 8 * E * lse.abs())
            mag = P @ V.abs()
            o_tol = (up + 2 * eps + (n + 16) * E) * mag + tiny(dt) * (seen.double() @ V.abs())
            o_tol = o_tol * (1 + 2 * u) + u * O.abs() + torch.where(empty, 0.0, tiny(dt))[:, None]
            r["out_tol"][q0:q1, h] = o_tol
            if grad is None:
                continue
            G = grad[q0:q1, h]
            m = q1 - q0
            D = (G * O).sum(-1, keepdim=True)
            dP = G @ V.T
            dS = torch.where(seen, P * (dP - D), 0.0)
            # of dP: a sum of d products; of D: the output's error and a sum
            dp_tol = (d + 2) * E * (G.abs() @ V.abs().T)
            d_tol = (G.abs() * o_tol).sum(-1, keepdim=True) + (d + 8) * E * (G.abs() * O.abs()).sum(-1, keepdim=True)
            spread = dS.abs() + P * (dp_tol + d_tol)
            ds_tol = (eps + 4 * E + up) * spread + P * (dp_tol + d_tol) * (1 + up)
            ds_tol = torch.where(seen, ds_tol, 0.0)
            # fp16 holds a score gradient, scaled to at most 2^15 per row or column, to 2^-24 of that and up
            low_q = tiny(dt) * 2.0 ** -14 * spread.amax(-1, keepdim=True) * seen
            low_k = tiny(dt) * 2.0 ** -14 * spread.amax(0, keepdim=True) * seen
            r["grad_q"][q0:q1, h] = scale * (dS @ K)
            t = scale * ((ds_tol + low_q + (n + 16) * E * spread) @ K.abs())
            r["grad_q_tol"][q0:q1, h] = t * (1 + u) + u * r["grad_q"][q0:q1, h].abs() + tiny(dt)
            r["grad_k"][k0:k1, g] += scale * (dS.T @ Q)
            r["grad_k_tol"][k0:k1, g] += scale * ((ds_tol + low_k + (m * group + 16) * E * spread).T @ Q.abs()) * (1 + u)
            r["grad_v"][k0:k1, g] += P.T @ G
            p_tol = (eps + up + (m * group + 16) * E) * P + tiny(dt) * 2.0 ** -14 * seen
            r["grad_v_tol"][k0:k1, g] += p_tol.T @ G.abs() * (1 + u)
    if grad is not None:
        for n in ("grad_k", "grad_v"):
            r[n + "_tol"] += u * r[n].abs() + tiny(dt)
    return r


def turn_factors(table, positions, rotary):
    """cos, sin [rows, 1, rotary / 2] of every pair."""
    table = table.double()
    axes = positions.shape[1]
    n = rotary // (2 * axes)
    got = []
    for part in (0, 1):
        cols = []
        for a in range(axes):
            p = positions[:, a].long()
            inside = (p >= 0) & (p < table.shape[0])
            row = table[p.clamp(0, table.shape[0] - 1), :n, part]
            cols.append(torch.where(inside[:, None], row, float("nan")))
        got.append(torch.cat(cols, 1)[:, None])
    return got


def pair_index(rotary, interleaved):
    at = torch.arange(rotary // 2)
    return (2 * at, 2 * at + 1) if interleaved else (at, at + rotary // 2)


def norm_rotary(x, weight, table, positions, rotary, interleaved, eps, grad=None):
    """out (and grad, grad_weight) of one tensor, with bounds.  The mean of d
    squares, its root and the products: (d + 12) e relative before the
    rotation; each rotated value: 3 e more of its two products."""
    dt, d = x.dtype, x.shape[2]
    u, rel = U[dt], (d + 12) * E
    x = x.double()
    if weight is not None:
        w = weight.double()
        inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    else:
        w, inv = torch.ones(d, dtype=torch.float64), torch.ones(1, dtype=torch.float64)
    y = x * inv * w
    out, mag = y.clone(), y.abs()
    if rotary:
        c, s = turn_factors(table, positions, rotary)
        a, b = pair_index(rotary, interleaved)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
        mag[..., a], mag[..., b] = (y[..., a] * c).abs() + (y[..., b] * s).abs(), (y[..., a] * s).abs() + (y[..., b] * c).abs()
    r = {"out": out, "out_tol": (rel + 3 * E) * mag * (1 + u) + u * out.abs() + tiny(dt)}
    if grad is None:
        return r
    go = grad.double()
    g, gm = go.clone(), go.abs()
    if rotary:
        g[..., a], g[..., b] = go[..., a] * c + go[..., b] * s, go[..., b] * c - go[..., a] * s
        gm[..., a], gm[..., b] = (go[..., a] * c).abs() + (go[..., b] * s).abs(), (go[..., b] * c).abs() + (go[..., a] * s).abs()
    if weight is None:
        r["grad"], r["grad_tol"] = g, 3 * E * gm * (1 + u) + u * g.abs() + tiny(dt)
        return r
    gw = g * w
    m = (gw * x).mean(-1, keepdim=True)
    r["grad"] = inv * (gw - x * inv * inv * m)
    mag = inv * (gm * w.abs() + x.abs() * inv * inv * (gm * w.abs() * x.abs()).mean(-1, keepdim=True))
    r["grad_tol"] = (3 * rel + (d + 16) * E) * mag * (1 + u) + u * r["grad"].abs() + tiny(dt)
    r["grad_weight"] = (g * x * inv).sum((0, 1))
    n = x.shape[0] * x.shape[1]
    r["grad_weight_tol"] = (rel + 8 * E + n * E) * (gm * x.abs() * inv).sum((0, 1))
    return r
