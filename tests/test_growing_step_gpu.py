"""selective_step where the state grows (A above 0): e^(dt A) alone passes
float32's range.  Against the 64-bit reference."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import sequence_reference as ref
from .test_sequence_gpu import DTYPES, check, gen, normal

pytestmark = pytest.mark.gpu


def test_step(gpu_device):
    """A state of 0 takes its input whatever the growth, also where an episode
    starts from a state that would not be; a tiny one grows to its value."""
    g = gen(73)
    N, ch, S = 3, 70, 5
    for dtype in DTYPES:
        t = {"u": normal(g, N, ch, dtype=dtype), "B": normal(g, N, 1, S, dtype=dtype),
             "C": normal(g, N, 1, S, dtype=dtype),
             "delta": torch.full((N, ch), 100.0, dtype=dtype, device="cuda"),
             "A": 1.0 + torch.rand(ch, S, generator=g, device="cuda") / 8}
        pool = torch.zeros(N, ch, S, device="cuda")
        pool[1] = normal(g, ch, S)
        pool[2] = 1e-30
        starts = torch.tensor([0, 1, 0], dtype=torch.uint8, device="cuda")
        rows = {k: v[..., None] if k != "A" else v for k, v in t.items()}
        want = ref.scan(**rows, state=pool.clone(), flags=starts[:, None])
        y = rl.selective_step(state=pool, flags=starts, **t)
        check(pool, want["final"], "state")
        if dtype != torch.float16:  # 1e-30 has grown past fp16's range
            check(y[:, :, None], want["y"], "y")
