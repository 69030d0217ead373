"""Infinite and NaN states of the gated recurrence: what they become, a NaN or an
infinity, stays one until an episode starts, whatever the decays multiply to, and so do
infinite gradients towards the row's begin; the single step does as the rows do."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_sequence_gpu import gen, normal

pytestmark = pytest.mark.gpu

# rows of 1, 4, 16 and 64 lanes, rows that a workgroup shares, chunked rows
SHAPES = [(5, 70, 6), (5, 17, 30), (300, 130, 100), (5, 30, 1100), (2, 60, 2600), (2, 3, 2051)]


def bads(T):
    """A step of the first row's that is bad, the second row's start, the bad gradient's."""
    return T // 4, T // 2, T - 2


@pytest.mark.parametrize("rate", [0.05, 3.0, 60.0, 300.0])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_states_stay(bad, rate, gpu_device):
    for N, D, T in SHAPES:
        for flagged in (False, True):
            print(f"gated {N}x{D}x{T} rate {rate} bad {bad} flags {flagged}", flush=True)
            g = gen(T)
            x, gates = normal(g, N, D, T), 0.1 * normal(g, N, 2 * D, T)
            # L = 8 softplus(decay) sigmoid(gate), about `rate` at every step
            decay = torch.full((D,), rate / 4, device="cuda").expm1().log() \
                if rate < 100 else torch.full((D,), rate / 4, device="cuda")
            at, start, back = bads(T)
            x[:2, :, at] = bad
            flags = None
            if flagged:
                flags = torch.zeros(N, T, dtype=torch.uint8, device="cuda")
                flags[1, start] = 1
            args = (x, gates[:, :D], gates[:, D:], decay)
            out, final, points = rl.gated_recurrence(*args, flags=flags, with_state=True,
                                                     with_checkpoints=True)
            ends = [T, start if flagged else T]
            for n in (0, 1):
                assert out[n, :, :at].isfinite().all()
                assert not out[n, :, at:ends[n]].isfinite().any()
                assert out[n, :, ends[n]:].isfinite().all()
                assert (final[n].isfinite() == (ends[n] < T)).all()
            assert out[2:].isfinite().all() and final[2:].isfinite().all()
            # the same from a state that is bad when the row begins
            state = normal(g, N, D)
            state[:2] = bad
            good = (torch.nan_to_num(x, 1.0, 1.0, -1.0), *args[1:])
            out, final, points = rl.gated_recurrence(*good, state=state, flags=flags,
                                                     with_state=True, with_checkpoints=True)
            for n in (0, 1):
                assert not out[n, :, :ends[n]].isfinite().any()
                assert out[n, :, ends[n]:].isfinite().all()
            # a bad gradient reaches every step before it, up to the start
            go = normal(g, N, D, T)
            go[:2, :, back] = bad
            points = rl.gated_recurrence(*good, flags=flags, with_checkpoints=True)[2]
            gx = rl.gated_recurrence_backward(go, *good, points, flags=flags).x
            begins = [0, start if flagged else 0]
            for n in (0, 1):
                assert not gx[n, :, begins[n]:back + 1].isfinite().any()
                assert gx[n, :, :begins[n]].isfinite().all()
                assert gx[n, :, back + 1:].isfinite().all()
            assert gx[2:].isfinite().all()


@pytest.mark.parametrize("rate", [0.05, 3.0, 300.0])
def test_bad_states_stay_in_single_steps(rate, gpu_device):
    g = gen(9)
    x, ig, dg = normal(g, 3, 40), normal(g, 3, 40), torch.zeros(3, 40, device="cuda")
    decay = torch.full((40,), rate / 4, device="cuda").expm1().log() if rate < 100 \
        else torch.full((40,), rate / 4, device="cuda")
    for bad in (float("nan"), float("inf")):
        state = normal(g, 3, 40)
        state[0], state[1] = bad, bad
        flags = torch.tensor([0, 1, 0], device="cuda", dtype=torch.uint8)
        out = rl.gated_step(x, ig, dg, decay, state, flags=flags)
        assert not out[0].isfinite().any() and not state[0].isfinite().any()
        assert out[1:].isfinite().all() and state[1:].isfinite().all()
