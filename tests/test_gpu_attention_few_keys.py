"""16-bit gradients of queries that see few keys, where dO v and D = dO out
nearly cancel: D has to be better than what the rounded output gives."""
import math

import pytest
import torch

import attention_reference as ref
from test_gpu_attention import DEV, DT, _near

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


def _gradients(q, k, v, grad, cu, dtype, **how):
    """64-bit gradients of q and k with bounds like attention_reference.py's,
    but for D: a sum in fp32 of the n probabilities times dP."""
    u, tiny, d = ref.U[dtype], ref.tiny(dtype), q.shape[2]
    q, k, v, grad = q.double(), k.double(), v.double(), grad.double()
    group, scale = q.shape[1] // k.shape[1], d ** -0.5
    gq, gk, tq, tk = (torch.zeros_like(x) for x in (q, k, q, k))
    for b in range(len(cu) - 1):
        s = slice(int(cu[b]), int(cu[b + 1]))
        n = s.stop - s.start
        seen = ref.visible(n, n, how.get("causal", False), how.get("window", (-1, -1)))
        for h in range(q.shape[1]):
            g = h // group
            Q, K, V, G = q[s, h], k[s, g], v[s, g], grad[s, h]
            score = torch.where(seen, (Q @ K.T) * scale, -math.inf)
            P = torch.softmax(score, -1)
            eps = (2 * d + 16) * E * torch.where(seen, (Q.abs() @ K.abs().T) * scale, 0.0).amax(-1, keepdim=True) + (n + 16 + 8 * math.log(n + 1)) * E
            dP = G @ V.T
            dp_tol = (d + 2) * E * (G.abs() @ V.abs().T)
            d_tol = (P * ((eps + (n + 8) * E) * dP.abs() + dp_tol)).sum(-1, keepdim=True)
            dS = P * (dP - (P * dP).sum(-1, keepdim=True))
            spread = dS.abs() + P * (dp_tol + d_tol)
            ds_tol = torch.where(seen, (eps + 4 * E + u) * spread + P * (dp_tol + d_tol) * (1 + u), 0.0)
            low = tiny * 2.0 ** -14 * seen
            gq[s, h] = scale * (dS @ K)
            tq[s, h] = scale * ((ds_tol + low * spread.amax(-1, keepdim=True) + (n + 16) * E * spread) @ K.abs()) * (1 + u)
            gk[s, g] += scale * (dS.T @ Q)
            tk[s, g] += scale * ((ds_tol + low * spread.amax(0, keepdim=True) + (n * group + 16) * E * spread).T @ Q.abs()) * (1 + u)
    return (gq, tq + u * gq.abs() + tiny), (gk, tk + u * gk.abs() + tiny)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 32), (4, 2, 72), (2, 1, 128), (1, 1, 16)])
@pytest.mark.parametrize("lengths,how", [([1, 2, 3, 17, 32, 33, 48, 64], dict()), ([5, 64, 31, 2], dict(causal=True)), ([300], dict(window=(15, 0))),
                                         ([3, 2, 4, 6], dict()), ([2, 130], dict(window=(8, 8)))])
def test_values_that_are_nearly_equal(sp, dtype, heads, kv_heads, dim, lengths, how):
    """Values 2^-6 around one vector: dO (v - out) is far below dO out."""
    g = torch.Generator().manual_seed(dim + len(lengths))
    dt, cu = DT[dtype], ref.offsets(lengths)
    n = int(cu[-1])
    q, grad = (torch.randn(n, heads, dim, generator=g).to(dt) for _ in range(2))
    k = torch.randn(n, kv_heads, dim, generator=g).to(dt)
    v = (torch.randn(1, kv_heads, dim, generator=g) + 2.0 ** -6 * torch.randn(n, kv_heads, dim, generator=g)).to(dt)
    dev, c = tuple(t.to(DEV) for t in (q, k, v)), cu.to(DEV)
    out, lse = sp.attention(*dev, c, return_lse=True, **how)
    gq, gk, _ = sp.attention_backward(grad.to(DEV), *dev, out, lse, c, **how)
    for name, got, (want, tol) in zip(("grad_q", "grad_k"), (gq, gk), _gradients(q, k, v, grad, cu, dt, **how)):
        _near(name, got, want, tol)
