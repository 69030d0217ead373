"""The norm's gradients over more channels than one launch of the weight's sums has
threads for: 2^28 channels at 16 threads each."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl

pytestmark = pytest.mark.gpu


def test_weight_gradient_of_many_channels(gpu_device):
    D = 2 ** 28 + 77
    x = torch.ones(1, D, device="cuda", dtype=torch.bfloat16)
    # -4 .. 3 in turn: a mean of about -1/2, and exact in bfloat16
    go = (torch.arange(D, device="cuda") % 8 - 4).to(torch.bfloat16)[None]
    w = torch.ones(D, device="cuda")
    grads = rl.rms_norm_backward(go, x, w, eps=1e-30)
    # x's root mean square is 1 up to the rounding of its sum: D / 256 / 8 serial terms a
    # thread, each rounding at most half a step of a sum of at most 2^20, so 2^17 2^-24 of it
    torch.testing.assert_close(grads.weight, go[0].float(), rtol=2.0 ** -7, atol=0)
    # the terms are multiples of one factor, and all channels are there
    one = grads.weight[:8].clone()
    whole = D // 8 * 8
    assert torch.equal(grads.weight[:whole].view(-1, 8), one.expand(whole // 8, 8))
    assert torch.equal(grads.weight[whole:], one[:D - whole])
