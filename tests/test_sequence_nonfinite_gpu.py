"""A NaN or infinity of the selective scan's state stays until an episode
starts: rows with episode flags keep one where their decay has underflowed to
0, as rows without flags do (0 times it is not 0)."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_sequence_gpu import gen, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2, 5, 4, 150), (20, 1026, 4, 70), (160, 510, 4, 13)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_underflown_decay_is_no_start(bad, shape, gpu_device):
    N, ch, S, T = shape
    g = gen(81)
    t = {"u": normal(g, N, ch, T), "delta": torch.full((N, ch, T), 50.0, device="cuda"),
         "A": torch.full((ch, S), -4.0, device="cuda"), "B": normal(g, N, 1, S, T),
         "C": normal(g, N, 1, S, T)}
    flags = torch.zeros(N, T, dtype=torch.uint8, device="cuda")
    flags[1, 9] = 1
    t["u"][:2, :, 4] = bad  # a is exp(-200), 0 in float32, at every step
    y, final, points = rl.selective_scan(**t, flags=flags, with_state=True, with_checkpoints=True)
    plain, plain_final, _ = rl.selective_scan(**t, with_state=True)
    assert not plain[0, :, 4:].isfinite().any() and not plain_final[0].isfinite().any()
    assert not y[0, :, 4:].isfinite().any() and not final[0].isfinite().any()
    assert not y[1, :, 4:9].isfinite().any()
    assert y[1, :, 9:].isfinite().all() and final[1].isfinite().all()
    go = normal(g, N, ch, T)
    go[:2, :, T - 2] = bad  # backward the same: up to the start, or the row's begin
    gr = rl.selective_scan_backward(go, **t, checkpoints=points, flags=flags)
    assert not gr.u[0].isfinite()[:, :T - 1].any()
    assert not gr.u[1].isfinite()[:, 9:T - 1].any() and gr.u[1, :, :4].isfinite().all()
