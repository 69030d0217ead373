"""The recurrent policy: what it computes step by step is what it learns from,
its gradients are the formula's, and it learns a task that needs memory."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_steps_and_rows_agree(gpu_device):
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    torch.manual_seed(3)
    policy = rp.RecurrentPolicy(5, 4, channels=20, states=6)
    env, state = rp.Recall(7), policy.new_state(7)
    rp.collect(policy, env, state, 4)  # the window starts inside episodes
    before = tuple(s.clone() for s in state)
    (obs, starts, action, logp, values, _, _), _ = rp.collect(policy, env, state, 21)
    logits, again = policy.rows(obs, starts, before)
    rows = logits.log_softmax(dim=1).gather(1, action[:, None]).squeeze(1)
    # every value is a few sums of at most 40 products of size ~1 with fp32
    # roundings, a different order in the two
    bound = 1e3 * torch.finfo(torch.float32).eps / 2
    assert (again - values).abs().max() < bound
    assert (rows - logp).abs().max() < bound


def test_gradients_against_differences(gpu_device):
    """A directional derivative of the rows' outputs in all parameters."""
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    torch.manual_seed(4)
    policy = rp.RecurrentPolicy(5, 4, channels=20, states=6)
    env, state = rp.Recall(7), policy.new_state(7)
    (obs, starts, *_), _ = rp.collect(policy, env, state, 30)
    zero = policy.new_state(7)
    weights = torch.randn(7, 5, 30, device="cuda")

    def value():
        logits, v = policy.rows(obs, starts, zero)
        return (torch.cat([logits, v[:, None]], dim=1) * weights).double().sum()

    loss = value()
    policy.zero_grad()
    loss.backward()
    params = list(policy.parameters())
    # along the gradient, so that the derivative is its norm
    norm = math.sqrt(sum(float(p.grad.double().pow(2).sum()) for p in params))
    step = 1e-3

    def at(t):
        with torch.no_grad():
            for p in params:
                p.add_(p.grad * (t / norm))
            out = float(value())
            for p in params:
                p.sub_(p.grad * (t / norm))
        return out

    slope = (at(step) - at(-step)) / (2 * step)
    # fp32 outputs (1050 of size ~1, 2^-22 relative each, as a random walk) over
    # 2e-3, and the third derivative times the step squared: well below 1%
    assert abs(slope - norm) < 0.01 * norm


def test_learns_to_recall(gpu_device):
    """Four cues: chance is 0.25; an agent without memory stays there."""
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    history = rp.train(updates=60)
    assert all(math.isfinite(r) for r in history)
    assert sum(history[:2]) / 2 < 0.4
    assert sum(history[-5:]) / 5 > 0.8
