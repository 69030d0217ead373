"""Autograd is told of what the calls write in place."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_sequence_gpu import gen, normal, scan_inputs

pytestmark = pytest.mark.gpu


def test_writes_in_place_are_noticed(gpu_device):
    """A tensor that autograd has saved and a call has changed since is refused
    by backward."""
    g = gen(94)

    def saved(like):
        x = like.detach()
        p = torch.ones_like(x, requires_grad=True)
        return x, (p * x).sum()

    x, loss = saved(normal(g, 50))
    rl.clip_grad_norm([x], 0.1)
    with pytest.raises(RuntimeError, match="in-?place"):
        loss.backward()
    x, loss = saved(normal(g, 50))
    rl.clip_grad_norm([x], float("inf"))  # only read
    loss.backward()
    src = normal(g, 50)
    x, loss = saved(normal(g, 50))
    rl.clip_grad_norm([src], 0.1, out=[x])
    with pytest.raises(RuntimeError, match="in-?place"):
        loss.backward()
    N, ch, S = 3, 6, 4
    pool, loss = saved(normal(g, N, ch, 3))
    rl.causal_conv_step(normal(g, N, ch), normal(g, ch, 4), None, pool)
    with pytest.raises(RuntimeError, match="in-?place"):
        loss.backward()
    t = {k: v[..., 0].contiguous() if k in ("u", "delta", "z", "B", "C") else v
         for k, v in scan_inputs(g, N, ch, S, 1, 1, torch.float32, True).items()}
    pool, loss = saved(normal(g, N, ch, S))
    rl.selective_step(state=pool, **t)
    with pytest.raises(RuntimeError, match="in-?place"):
        loss.backward()
    for call in (lambda out: rl.causal_conv(normal(g, N, ch, 9), normal(g, ch, 4), out=out),
                 lambda out: rl.selective_scan(y=out, **scan_inputs(g, N, ch, S, 9, 1,
                                                                    torch.float32, True))):
        out, loss = saved(normal(g, N, ch, 9))
        call(out)
        with pytest.raises(RuntimeError, match="in-?place"):
            loss.backward()
