"""The residual stack of gated recurrences, with norm, recurrence, single steps and
beams as they are used together: what it computes step by step is what it learns
from, its gradients are the formula's, it trains, and its plans are the likeliest
sequences of all."""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def plain_rows(policy, obs, starts, state):
    """GatedPolicy.rows from the formulas in float64, step by step."""
    def d(t):
        return t.double()

    new, stream = d(policy.w_in) @ d(obs), 0.0

    def normed(s, w):
        return s / (s.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * d(w)[:, None]

    for i in range(len(policy.decays)):
        stream = stream + new
        x, ig, dg = (d(policy.w_gates[i]) @ normed(stream, policy.norms[i])).split(
            policy.channels, dim=1)
        ig = torch.sigmoid(ig + d(policy.input_biases[i])[:, None])
        dg = torch.sigmoid(dg + d(policy.decay_biases[i])[:, None])
        a = torch.exp(-8 * torch.nn.functional.softplus(d(policy.decays[i]))[:, None] * dg)
        b = torch.sqrt(1 - a * a) * ig * x
        h, hs = d(state[i]), []
        for t in range(obs.shape[2]):
            h = a[:, :, t] * torch.where(starts[:, t:t + 1] != 0, 0.0, h) + b[:, :, t]
            hs.append(h)
        new = d(policy.w_blocks[i]) @ torch.stack(hs, 2)
    out = d(policy.w_out) @ normed(stream + new, policy.norms[-1])
    return out[:, :-1], out[:, -1]


def window(policy, rp, envs, T):
    env, state = rp.Recall(envs), policy.new_state(envs)
    rp.collect(policy, env, state, 4)  # the window starts inside episodes
    before = tuple(s.clone() for s in state)
    return before, rp.collect(policy, env, state, T)[0]


def test_steps_rows_and_the_formulas_agree(gpu_device):
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    torch.manual_seed(5)
    policy = rp.GatedPolicy(5, 4, channels=20)
    before, (obs, starts, action, logp, values, _, _) = window(policy, rp, 7, 33)
    want_logits, want_value = plain_rows(policy, obs, starts, before)
    logits, value = policy.rows(obs, starts, before)
    # each value is a few sums of at most 20 products of size ~1 with fp32 roundings
    bound = 1e3 * torch.finfo(torch.float32).eps / 2
    assert (logits - want_logits).abs().max() < bound
    assert (value - want_value).abs().max() < bound
    assert (values - want_value).abs().max() < bound
    want = want_logits.log_softmax(dim=1).gather(1, action[:, None]).squeeze(1)
    assert (logp - want).abs().max() < bound


def test_gradients_are_the_formulas(gpu_device):
    """Of all parameters, against automatic differentiation in float64."""
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    torch.manual_seed(6)
    policy = rp.GatedPolicy(5, 4, channels=20)
    before, (obs, starts, *_) = window(policy, rp, 7, 30)
    weights = torch.randn(7, 5, 30, device="cuda")

    def grads(rows):
        logits, v = rows(obs, starts, before)
        loss = (torch.cat([logits, v[:, None]], dim=1) * weights).sum()
        return torch.autograd.grad(loss, list(policy.parameters()))

    got = grads(policy.rows)
    want = grads(lambda *a: plain_rows(policy, *a))
    for (name, _), g, w in zip(policy.named_parameters(), got, want):
        # sums of at most 210 terms, each of a chain of ~20 products and sums
        bound = 230 * 20 * 2.0 ** -24 * float(w.abs().max()) + 1e-4 * float(w.abs().mean())
        assert (g - w).abs().max() <= bound, name


def test_trains(gpu_device):
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    history = rp.train(updates=4, num_envs=64, core="gated")
    assert len(history) == 4 and all(math.isfinite(r) for r in history)


@pytest.mark.parametrize("beams", [16, 1])
def test_plans(beams, gpu_device):
    """With 16 beams of 4 actions no prefix of a three-step plan is lost."""
    from linear_recurrence_scan_row_amd import recurrent_policy as rp
    torch.manual_seed(7)
    policy = rp.GatedPolicy(5, 4, channels=20)
    with torch.no_grad():
        policy.w_out.mul_(30)  # actions of different likelihoods
    N, steps = 3, 3
    first = torch.nn.functional.one_hot(torch.arange(N, device="cuda") % 4, 5).float()

    def model(actions):
        return torch.nn.functional.one_hot(actions, 5).float()

    found, scores = rp.plan(policy, first, model, steps, beams=beams)
    assert found.shape == (N, beams, steps) and scores.shape == (N, beams)
    every = torch.tensor(list(itertools.product(range(4), repeat=steps)), device="cuda")
    for n in range(N):
        obs = torch.cat([first[n].expand(len(every), 1, 5), model(every[:, :-1])], 1)
        starts = torch.zeros(len(every), steps, dtype=torch.uint8, device="cuda")
        zero = tuple(torch.zeros(len(every), 20, device="cuda") for _ in policy.decays)
        logits, _ = plain_rows(policy, obs.transpose(1, 2).contiguous(), starts, zero)
        total = logits.log_softmax(1).gather(1, every[:, None]).sum((1, 2))
        index = (found[n] * torch.tensor([16, 4, 1], device="cuda")).sum(1)
        # each beam's score is its sequence's
        assert (total[index] - scores[n]).abs().max() < 1e-4
        if beams == 16:
            order = total.sort(descending=True).values[:beams]
            assert (order - scores[n]).abs().max() < 1e-4
            assert len(set(index.tolist())) == beams
        else:
            # greedy: the likeliest action at every step
            for t in range(steps):
                same = (every[:, :t] == found[n, 0, :t]).all(1)
                now = logits[same, :, t].mean(0)
                assert int(now.argmax()) == int(found[n, 0, t])
