"""The norm's 8-bit output over no channels: its scales are written (0), in rows and in
single steps, within a row's length and past it."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(3, 0, 9), (3, 0), (1, 0, 1), (70, 0, 30000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_scales_of_no_channels_are_written(shape, gpu_device):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(shape, device="cuda", dtype=dtype)
        given = torch.full((*shape[:1], *shape[2:]), 7.0, device="cuda")
        lengths = torch.full(shape[:1], 1, device="cuda", dtype=torch.int32)
        for kw in ({}, {"residual": x}, {"lengths": lengths}):
            given.fill_(7.0)
            q, scale, _ = rl.rms_norm_8bit(x, scale=given, **kw)
            assert scale is given and q.shape == shape
            assert not scale.any()
