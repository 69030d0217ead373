"""clip_grad_norm where float32 does not hold the scale."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("max_norm", [1e-2, 1e-5, 1e-8])
def test_scales_below_float32(max_norm, dtype, gpu_device):
    """Gradients next to the type's largest value and a small max_norm: the
    scale is subnormal in float32 (1e-2), or 0 (1e-5 and below); the results
    are not."""
    n = 1 << 20
    t = torch.full((n,), 3e38, device="cuda", dtype=dtype)
    t[::2] = -2.5e38
    value = t.double()
    norm = float(value.square().sum().sqrt())
    out = torch.empty_like(t)
    assert rl.clip_grad_norm([t], max_norm, out=[out]).item() == pytest.approx(norm, rel=1e-10)
    want = value * (max_norm / (norm + 1e-6))
    # the scale's and the product's roundings, and the type's
    tol = want.abs() * (3 * 2.0 ** -24 + torch.finfo(dtype).eps / 2)
    assert bool(((out.double() - want).abs() <= tol).all())
    rl.clip_grad_norm([t], max_norm)
    assert torch.equal(t, out)
