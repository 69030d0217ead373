"""A recurrent policy trained with PPO on this library's calls end to end:

    python -m linear_recurrence_scan_row_amd.recurrent_policy

The core is the usual selective state space block: a projection to u and a gate
z, the short causal convolution, the scan with dt, B and C computed from u, and
two heads on its output.  It acts one step at a time (causal_conv_step,
selective_step, states updated in place) and learns from the whole window at
once (causal_conv and selective_scan over rows with episode starts, and their
backward calls); the advantages come from gae_stats, the surrogate and its
gradient from ppo_clip_loss, and clip_grad_norm bounds the step.  The matrix
products between them are torch's.

With --core gated the policy is a residual stack of gated recurrences instead:
rms_norm adds each block's output to the stream and norms it, gated_recurrence and
gated_step carry the memory, and plan() searches for its likeliest sequences of
actions with beam_select and beam_reorder, the states of all beams in pools.

The task cannot be solved without memory: a cue is shown at an episode's first
step, and its last step is rewarded if the action names it.
"""
from __future__ import annotations

import argparse

import torch
from torch.autograd.function import once_differentiable

from . import (beam_reorder, beam_select, causal_conv, causal_conv_backward, causal_conv_step,
               clip_grad_norm, gae_stats, gated_recurrence, gated_recurrence_backward, gated_step,
               ppo_clip_loss, rms_norm, rms_norm_backward, selective_scan,
               selective_scan_backward, selective_step)


class _Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, flags):
        ctx.save_for_backward(x, weight, bias, state, flags)
        return causal_conv(x, weight, bias, state=state, flags=flags)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, weight, bias, state, flags = ctx.saved_tensors
        g = causal_conv_backward(grad.contiguous(), x, weight, bias, state=state, flags=flags)
        return g.x, g.weight, g.bias, g.state, None


class _Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, state, flags):
        y, _, checkpoints = selective_scan(u, delta, A, B, C, D, z, delta_bias, state=state,
                                           flags=flags, with_checkpoints=True)
        ctx.save_for_backward(u, delta, A, B, C, checkpoints, D, z, delta_bias, state, flags)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        B, C = ctx.saved_tensors[3:5]
        g = selective_scan_backward(grad.contiguous(), *ctx.saved_tensors)
        return (g.u, g.delta, g.A, g.B.view(B.shape), g.C.view(C.shape), g.D, g.z, g.delta_bias,
                g.state, None)


class _Norm(torch.autograd.Function):
    """(normed, s) of s = x + residual."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        out, s = rms_norm(x, weight, residual)
        ctx.save_for_backward(s, weight)
        return out, s

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, grad_sum):
        s, weight = ctx.saved_tensors
        g = rms_norm_backward(grad.contiguous(), s, weight, grad_sum=grad_sum.contiguous())
        return g.x, g.x, g.weight


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, input_gate, decay_gate, decay, input_bias, decay_bias, state, flags):
        h, _, checkpoints = gated_recurrence(x, input_gate, decay_gate, decay, input_bias,
                                             decay_bias, state=state, flags=flags,
                                             with_checkpoints=True)
        ctx.save_for_backward(x, input_gate, decay_gate, decay, checkpoints, input_bias,
                              decay_bias, state, flags)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        *inputs, state, flags = ctx.saved_tensors
        g = gated_recurrence_backward(grad.contiguous(), *inputs, state=state, flags=flags)
        return (g.x, g.input_gate, g.decay_gate, g.decay, g.input_bias, g.decay_bias, g.state,
                None)


class RecurrentPolicy(torch.nn.Module):
    """Logits and value from one selective state space block (float32)."""

    def __init__(self, observations, actions, channels=64, states=16, rank=4, width=4,
                 device="cuda"):
        super().__init__()
        self.sizes = (channels, states, rank)

        def matrix(rows, cols, scale=1.0):
            w = torch.randn(rows, cols, device=device) * (scale / cols ** 0.5)
            return torch.nn.Parameter(w)

        self.w_in = matrix(2 * channels, observations, observations ** 0.5)
        self.conv_weight = matrix(channels, width)
        self.conv_bias = torch.nn.Parameter(torch.zeros(channels, device=device))
        self.w_scan = matrix(rank + 2 * states, channels)
        self.w_delta = matrix(channels, rank)
        # dt between 0.01 and 0.3 at the start: softplus(bias) = dt
        dt = torch.logspace(-2, -0.5, channels, device=device)
        self.delta_bias = torch.nn.Parameter(torch.log(torch.expm1(dt)))
        self.a_log = torch.nn.Parameter(
            torch.arange(1, states + 1, device=device).float().log().repeat(channels, 1))
        self.skip = torch.nn.Parameter(torch.ones(channels, device=device))
        self.w_out = matrix(actions + 1, channels, 0.1)

    def new_state(self, num_envs):
        """What acting carries from step to step: the convolution's inputs and
        the scan's states."""
        channels, states, _ = self.sizes
        dev = self.w_in.device
        return (torch.zeros(num_envs, channels, self.conv_weight.shape[1] - 1, device=dev),
                torch.zeros(num_envs, channels, states, device=dev))

    @torch.no_grad()
    def step(self, obs, starts, state):
        """One step of every environment: obs [num_envs, observations], starts
        [num_envs] marks new episodes; state is updated in place."""
        channels, states, rank = self.sizes
        conv_state, scan_state = state
        x, z = (obs @ self.w_in.t()).split(channels, dim=1)
        u = causal_conv_step(x, self.conv_weight, self.conv_bias, conv_state, flags=starts)
        low, B, C = (u @ self.w_scan.t()).split((rank, states, states), dim=1)
        y = selective_step(u, low @ self.w_delta.t(), -self.a_log.exp(), B, C, scan_state,
                           self.skip, z, self.delta_bias, flags=starts)
        out = y @ self.w_out.t()
        return out[:, :-1], out[:, -1]

    def rows(self, obs, starts, state):
        """The same over a window: obs [num_envs, observations, T], starts
        [num_envs, T], state as it was when the window began."""
        channels, states, rank = self.sizes
        conv_state, scan_state = state
        x, z = torch.matmul(self.w_in, obs).split(channels, dim=1)
        u = _Conv.apply(x, self.conv_weight, self.conv_bias, conv_state, starts)
        low, B, C = torch.matmul(self.w_scan, u).split((rank, states, states), dim=1)
        y = _Scan.apply(u, torch.matmul(self.w_delta, low), -self.a_log.exp(), B, C, self.skip,
                        z, self.delta_bias, scan_state, starts)
        out = torch.matmul(self.w_out, y)
        return out[:, :-1], out[:, -1]


class GatedPolicy(torch.nn.Module):
    """Logits and value from a residual stack of gated recurrences (float32)."""

    def __init__(self, observations, actions, channels=64, blocks=2, device="cuda"):
        super().__init__()
        self.channels = channels

        def matrix(rows, cols, scale=1.0):
            w = torch.randn(rows, cols, device=device) * (scale / cols ** 0.5)
            return torch.nn.Parameter(w)

        def each(make):
            return torch.nn.ParameterList([make() for _ in range(blocks)])

        def constant(value, n=channels):
            return torch.nn.Parameter(torch.full((n,), value, device=device))

        self.w_in = matrix(channels, observations, observations ** 0.5)
        self.norms = torch.nn.ParameterList([constant(1.0) for _ in range(blocks + 1)])
        self.w_gates = each(lambda: matrix(3 * channels, channels))
        # a between 0.5 and 0.99 with an open decay gate: 8 softplus(decay) = -log(a)
        slow = -torch.logspace(-0.3, -0.005, channels, device=device).log() / 8
        self.decays = each(lambda: torch.nn.Parameter(torch.log(torch.expm1(slow))))
        self.input_biases = each(lambda: constant(0.0))
        self.decay_biases = each(lambda: constant(0.0))
        self.w_blocks = each(lambda: matrix(channels, channels, 0.5))
        self.w_out = matrix(actions + 1, channels, 0.1)

    def new_state(self, num_envs):
        """What acting carries from step to step: each block's states."""
        return tuple(torch.zeros(num_envs, self.channels, device=self.w_in.device)
                     for _ in self.decays)

    @torch.no_grad()
    def step(self, obs, starts, state, slots=None):
        """One step of every environment: obs [num_envs, observations], starts
        [num_envs] marks new episodes (or None); state, at the places that slots give,
        is updated in place."""
        new, stream = obs @ self.w_in.t(), None
        for norm, w, decay, ib, db, w_block, pool in zip(
                self.norms, self.w_gates, self.decays, self.input_biases, self.decay_biases,
                self.w_blocks, state):
            y, total = rms_norm(new, norm, stream)
            stream = new if stream is None else total
            x, ig, dg = (y @ w.t()).split(self.channels, dim=1)
            new = gated_step(x, ig, dg, decay, pool, ib, db, slots=slots,
                             flags=starts) @ w_block.t()
        out = rms_norm(new, self.norms[-1], stream)[0] @ self.w_out.t()
        return out[:, :-1], out[:, -1]

    def rows(self, obs, starts, state):
        """The same over a window: obs [num_envs, observations, T], starts
        [num_envs, T], state as it was when the window began."""
        new = torch.matmul(self.w_in, obs)
        stream = torch.zeros_like(new)
        for norm, w, decay, ib, db, w_block, begin in zip(
                self.norms, self.w_gates, self.decays, self.input_biases, self.decay_biases,
                self.w_blocks, state):
            y, stream = _Norm.apply(new, stream, norm)
            x, ig, dg = torch.matmul(w, y).split(self.channels, dim=1)
            new = torch.matmul(w_block, _Gated.apply(x, ig, dg, decay, ib, db, begin, starts))
        out = torch.matmul(self.w_out, _Norm.apply(new, stream, self.norms[-1])[0])
        return out[:, :-1], out[:, -1]


@torch.no_grad()
def plan(policy, obs, model, steps, beams=4):
    """The likeliest sequences of actions of a GatedPolicy from new episodes: obs
    [N, observations] is what each episode begins with, and model(actions), actions
    [N * beams] int64, gives the observations that follow.  Returns the actions
    [N, beams, steps] and their log probabilities [N, beams], the likeliest first.
    The beams' states and their actions so far lie in pools that beam_reorder keeps in
    order."""
    N = len(obs)
    dev = obs.device
    pools = policy.new_state(N * beams)
    taken = torch.zeros(N * beams, steps, dtype=torch.int64, device=dev)
    slots = torch.arange(N * beams, dtype=torch.int32, device=dev).view(N, beams)
    # at first the beams of an episode are alike, so one of them counts
    scores = torch.full((N, beams), -float("inf"), device=dev)
    scores[:, 0] = 0.0
    obs = obs.repeat_interleave(beams, 0)
    for t in range(steps):
        logits, _ = policy.step(obs, None, pools, slots=slots.view(-1))
        choice = beam_select(logits.view(N, beams, -1), scores)
        slots = beam_reorder([*pools, taken], slots, choice.parents)
        scores, actions = choice.scores, choice.tokens.view(-1).long()
        taken[slots.view(-1).long(), t] = actions
        obs = model(actions)
    return taken[slots.view(-1).long()].view(N, beams, steps), scores


class Recall:
    """Environments whose observation is the cue (one-hot) at an episode's first
    step, zero after it, and a last entry that is 1 at its last step."""

    def __init__(self, num_envs, cues=4, steps=6, device="cuda"):
        self.cues, self.steps = cues, steps
        self.cue = torch.randint(cues, (num_envs,), device=device)
        self.at = torch.zeros(num_envs, dtype=torch.long, device=device)

    def observe(self):
        obs = torch.zeros(len(self.at), self.cues + 1, device=self.at.device)
        first = self.at == 0
        obs[:, :-1] = torch.nn.functional.one_hot(self.cue, self.cues) * first[:, None]
        obs[:, -1] = self.at == self.steps - 1
        return obs, first.to(torch.uint8)

    def act(self, action):
        last = self.at == self.steps - 1
        reward = (last & (action == self.cue)).float()
        self.at = torch.where(last, 0, self.at + 1)
        self.cue = torch.where(last, torch.randint_like(self.cue, self.cues), self.cue)
        return reward, last.to(torch.uint8)


def collect(policy, env, state, T):
    """A window of T steps: observations, starts, actions, their log
    probabilities, values, rewards, terminations, and the value after it."""
    steps = []
    for _ in range(T):
        obs, starts = env.observe()
        logits, value = policy.step(obs, starts, state)
        logp = logits.log_softmax(dim=1)
        action = torch.multinomial(logp.exp(), 1).squeeze(1)
        reward, done = env.act(action)
        steps.append((obs, starts, action, logp.gather(1, action[:, None]).squeeze(1), value,
                      reward, done))
    window = [torch.stack(x, dim=-1) for x in zip(*steps)]
    ahead = tuple(s.clone() for s in state)  # the next window's first step is not taken yet
    bootstrap = policy.step(*env.observe(), ahead)[1].contiguous()
    return window, bootstrap


def update(policy, optimizer, window, bootstrap, state, epochs=2, gamma=0.95, lam=0.95,
           value_weight=0.5, max_norm=0.5):
    """PPO on one window; returns the norm of the last epoch's gradient."""
    obs, starts, action, logp_old, values, rewards, done = window
    advantages, returns, stats = gae_stats(rewards, values, done, bootstrap=bootstrap,
                                           gamma=gamma, lam=lam)
    for _ in range(epochs):
        logits, value = policy.rows(obs, starts, state)
        logp = logits.log_softmax(dim=1).gather(1, action[:, None]).squeeze(1)
        _, grad_logp = ppo_clip_loss(advantages, logp.detach().contiguous(), logp_old, stats)
        grad_value = value_weight * (value.detach() - returns) / returns.numel()
        optimizer.zero_grad(set_to_none=True)
        torch.autograd.backward([logp, value], [grad_logp, grad_value])
        norm = clip_grad_norm([p.grad for p in policy.parameters()], max_norm)
        optimizer.step()
    return norm


CORES = {"selective": RecurrentPolicy, "gated": GatedPolicy}


def train(updates=60, num_envs=256, T=48, lr=1e-2, seed=0, report=None, core="selective"):
    """Mean reward per episode of each window."""
    torch.manual_seed(seed)
    env = Recall(num_envs)
    policy = CORES[core](env.cues + 1, env.cues)
    optimizer = torch.optim.Adam(policy.parameters(), lr=lr)
    state = policy.new_state(num_envs)
    history = []
    for i in range(updates):
        before = tuple(s.clone() for s in state)
        window, bootstrap = collect(policy, env, state, T)
        norm = update(policy, optimizer, window, bootstrap, before)
        rewards, done = window[-2:]
        history.append(float(rewards.sum() / done.sum()))
        if report is not None:
            report(i, history[-1], float(norm))
    return history


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--updates", type=int, default=60)
    parser.add_argument("--envs", type=int, default=256)
    parser.add_argument("--steps", type=int, default=48, help="steps of a window")
    parser.add_argument("--core", choices=sorted(CORES), default="selective")
    args = parser.parse_args()
    train(args.updates, args.envs, args.steps, core=args.core, report=lambda i, r, norm: print(
        f"update {i:3d}  reward per episode {r:.3f}  gradient norm {norm:.3f}", flush=True))


if __name__ == "__main__":
    main()
