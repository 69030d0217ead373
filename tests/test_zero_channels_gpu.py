"""selective_scan_backward without channels: B and C have no one to answer to,
and their gradients are 0."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_gradients_of_no_channels(dtype, gpu_device):
    N, S, T, G = 2, 3, 50, 2
    x = torch.zeros(N, 0, T, device="cuda", dtype=dtype)
    A = torch.zeros(0, S, device="cuda")
    B = torch.ones(N, G, S, T, device="cuda", dtype=dtype)
    # memory that torch hands out next is not 0
    used = [torch.full_like(B, float("nan")) for _ in range(8)]
    del used
    y, final, points = rl.selective_scan(x, x, A, B, B, with_state=True, with_checkpoints=True)
    assert y.shape == x.shape and final.shape == (N, 0, S)
    grads = rl.selective_scan_backward(x, x, x, A, B, B, points)
    for grad in (grads.B, grads.C):
        assert grad.shape == B.shape and grad.dtype == dtype and not grad.any()
    assert grads.u.shape == x.shape and grads.A.shape == A.shape
