"""The norm's 8-bit output of dense rows goes into an 8-bit matrix product as it is, its
scales with it; of rows over time, as a transposed copy."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_sequence_gpu import gen, normal

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not hasattr(torch, "_scaled_mm"),
                                                  reason="torch without an 8-bit product")]


def product(q, scale, w8, w_scale):
    return torch._scaled_mm(q, w8.t(), scale_a=scale, scale_b=w_scale, out_dtype=torch.bfloat16)


def test_8bit_rows_go_into_a_product(gpu_device):
    g = gen(1)
    M, D, F = 64, 512, 256
    w = normal(g, F, D)
    w_scale = w.abs().amax(1) / 448
    w8 = (w / w_scale[:, None]).to(torch.float8_e4m3fn)
    rows = normal(g, 2, D, M // 2, dtype=torch.bfloat16)
    dense = rows.transpose(1, 2).reshape(M, D)
    q, scale, _ = rl.rms_norm_8bit(dense)
    y = product(q, scale[:, None], w8, w_scale[None])
    a, b = q.double().cpu() * scale.double().cpu()[:, None], (w8.float() * w_scale[:, None]).double().cpu()
    want = a @ b.t()
    # 512 sums and two scales in float32, and one rounding to bfloat16
    bound = want.abs() * 2.0 ** -8 + (D + 4) * 2.0 ** -23 * (a.abs() @ b.abs().t())
    assert ((y.double().cpu() - want).abs() <= bound).all()
    # rows over time: the same codes, a step's channels apart
    qt, st, _ = rl.rms_norm_8bit(rows)
    # another order of the sums: their last bits, and codes at a border
    torch.testing.assert_close(st.reshape(M), scale, rtol=2.0 ** -18, atol=0)
    turned = qt.transpose(1, 2).reshape(M, D)
    y = product(turned, st.reshape(M, 1), w8, w_scale[None])
    a = turned.double().cpu() * st.double().cpu().reshape(M, 1)
    bound = bound + (a @ b.t() - want).abs() * (1 + 2.0 ** -8)
    assert ((y.double().cpu() - want).abs() <= bound).all()
