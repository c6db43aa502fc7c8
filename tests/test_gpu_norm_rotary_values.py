"""The rotation over values that are not finite: what is not rotated is
copied."""
import math

import pytest
import torch

from test_gpu_norm_rotary import DEV, DT, _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,axes,rotary", [(16, 3, 12), (24, 2, 16), (32, 3, 24), (64, 1, 2), (48, 1, 30), (128, 1, 64)])
def test_values_past_the_rotation_are_copied(sp, dtype, interleaved, dim, axes, rotary):
    """Without a norm the elements past rotary_dim come out bit for bit, and an
    infinity or NaN among them reaches no other element; in the gradient too."""
    x, _, grads, positions, table = _case(dim, 70, 3, 2, dim, dtype, axes, rotary)
    td, pd = table.to(DEV), positions.to(DEV)
    how = dict(rotary_dim=rotary, interleaved=interleaved)

    def forward(t):
        return torch.cat(sp.norm_rotary(t[:, :3], t[:, 3:5], None, None, td, pd, **how), 1)

    def backward(t):
        return torch.cat(sp.norm_rotary_backward(t[:, :3], t[:, 3:], xd[:, :3], xd[:, 3:5], None, None, td, pd, **how)[:2], 1)

    xd = x.to(DEV)
    for call, given in ((forward, xd[:, :5]), (backward, grads.to(DEV))):
        clean = call(given)
        bad = given.clone()
        for i, value in enumerate((math.inf, -math.inf, math.nan, -0.0)):
            bad[7 * i:70:5, :, rotary + (i * 3) % (dim - rotary)] = value
        got = call(bad)
        bits = torch.int32 if dtype == "f32" else torch.int16
        assert torch.equal(got[..., :rotary], clean[..., :rotary])
        same = (got[..., rotary:].view(bits) == bad[..., rotary:].contiguous().view(bits)) | (got[..., rotary:].isnan() & bad[..., rotary:].isnan())
        assert bool(same.all())
