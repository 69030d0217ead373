"""The 64-bit reference of the sequence operators (sequence_reference.py): its
gradients against automatic differentiation of the same definitions written
without a backward formula, and against differences; its episode rules against
rows cut by hand.  CPU only."""
import pytest
import torch

from . import sequence_reference as ref

pytestmark = []


def rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def auto_conv(x, w, bias, state, starts, ends, over, silu):
    """out and final state, with torch operations that differentiate."""
    N, D, T = x.shape
    W = w.shape[1]
    outs, finals = [], []
    for n in range(N):
        window = [state[n, :, i] if state is not None else torch.zeros(D, dtype=x.dtype)
                  for i in range(W - 1)]
        row = []
        for t in range(T):
            if t >= ends[n]:
                row.append(torch.zeros(D, dtype=x.dtype))
                continue
            if starts[n, t]:
                window = [torch.zeros_like(v) for v in window]
            window = window + [x[n, :, t]]
            pre = bias + sum(w[:, k] * window[k] for k in range(W))
            row.append(pre / (1 + torch.exp(-pre)) if silu else pre)
            window = window[1:]
        if over[n]:
            window = [torch.zeros_like(v) for v in window]
        outs.append(torch.stack(row, 1) if T else x[n])
        finals.append(torch.stack(window, 1))
    return torch.stack(outs), torch.stack(finals)


def auto_scan(u, delta, A, B, C, D, z, bias, h0, starts, ends, over, softplus):
    N, ch, T = u.shape
    G = B.shape[1]
    ys, hs = [], []
    for n in range(N):
        h = h0[n]
        row = []
        for t in range(T):
            if t >= ends[n]:
                row.append(torch.zeros(ch, dtype=u.dtype))
                continue
            if starts[n, t]:
                h = torch.zeros_like(h)
            dt = delta[n, :, t] + bias
            dt = torch.log1p(torch.exp(dt)) if softplus else dt
            b = B[n, :, :, t].repeat_interleave(ch // G, 0)
            c = C[n, :, :, t].repeat_interleave(ch // G, 0)
            h = torch.exp(dt[:, None] * A) * h + (dt * u[n, :, t])[:, None] * b
            y = (h * c).sum(1) + D * u[n, :, t]
            row.append(y * z[n, :, t] / (1 + torch.exp(-z[n, :, t])))
        ys.append(torch.stack(row, 1))
        hs.append(torch.zeros_like(h) if over[n] else h)
    return torch.stack(ys), torch.stack(hs)


def flags_and_lengths(g, N, T, which):
    flags = (torch.rand(N, T, generator=g) < 0.2).to(torch.uint8) if "flags" in which else None
    lengths = torch.randint(0, T + 1, (N,), generator=g).to(torch.int32) \
        if "lengths" in which else None
    return flags, lengths


@pytest.mark.parametrize("which", ["", "flags", "lengths", "flags lengths"])
@pytest.mark.parametrize("convention", [ref.ON_START, ref.AFTER_DONE])
@pytest.mark.parametrize("W,silu", [(2, True), (4, True), (3, False)])
def test_conv_gradients_against_autograd(which, convention, W, silu):
    g = torch.Generator().manual_seed(5 + W)
    N, D, T = 4, 3, 9
    x, w, b, s = rand(g, N, D, T), rand(g, D, W), rand(g, D), rand(g, N, D, W - 1)
    flags, lengths = flags_and_lengths(g, N, T, which)
    go, gf = rand(g, N, D, T), rand(g, N, D, W - 1)
    r = ref.conv(x, w, b, s, flags, convention, lengths, silu, go, gf)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, s)]
    starts, ends = ref.starts_of(flags, convention, N, T), ref.ends_of(lengths, N, T)
    over = ref.over_of(flags, convention, ends, N)
    out, final = auto_conv(*leaves, starts, ends, over, silu)
    torch.testing.assert_close(r["out"][0], out.detach(), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(r["final"][0], final.detach(), rtol=0, atol=0)
    ((out * go).sum() + (final * gf).sum()).backward()
    for name, leaf in zip(("x", "weight", "bias", "state"), leaves):
        torch.testing.assert_close(r[name][0], leaf.grad, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("which", ["", "flags", "lengths", "flags lengths"])
@pytest.mark.parametrize("convention", [ref.ON_START, ref.AFTER_DONE])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_against_autograd(which, convention, softplus):
    g = torch.Generator().manual_seed(7)
    N, ch, S, T, G = 3, 4, 3, 8, 2
    t = {"u": rand(g, N, ch, T), "delta": rand(g, N, ch, T).abs(), "A": -rand(g, ch, S).abs(),
         "B": rand(g, N, G, S, T), "C": rand(g, N, G, S, T), "D": rand(g, ch),
         "z": rand(g, N, ch, T), "delta_bias": rand(g, ch), "state": rand(g, N, ch, S)}
    flags, lengths = flags_and_lengths(g, N, T, which)
    go, gf = rand(g, N, ch, T), rand(g, N, ch, S)
    r = ref.scan(**t, flags=flags, convention=convention, lengths=lengths, softplus=softplus,
                 grad_y=go, grad_final=gf)
    leaf = {k: v.clone().requires_grad_() for k, v in t.items()}
    starts, ends = ref.starts_of(flags, convention, N, T), ref.ends_of(lengths, N, T)
    over = ref.over_of(flags, convention, ends, N)
    y, final = auto_scan(*(leaf[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias",
                                             "state")), starts, ends, over, softplus)
    torch.testing.assert_close(r["y"][0], y.detach(), rtol=1e-11, atol=1e-12)
    torch.testing.assert_close(r["final"][0], final.detach(), rtol=1e-11, atol=1e-12)
    ((y * go).sum() + (final * gf).sum()).backward()
    for name in t:
        torch.testing.assert_close(r[name][0], leaf[name].grad, rtol=1e-10, atol=1e-11)


def test_scan_gradients_against_differences():
    g = torch.Generator().manual_seed(9)
    N, ch, S, T = 2, 3, 2, 5
    t = {"u": rand(g, N, ch, T), "delta": rand(g, N, ch, T), "A": -rand(g, ch, S).abs(),
         "B": rand(g, N, 1, S, T), "C": rand(g, N, 1, S, T), "D": rand(g, ch),
         "z": rand(g, N, ch, T), "delta_bias": rand(g, ch), "state": rand(g, N, ch, S)}
    flags = torch.tensor([[0, 0, 1, 0, 0], [1, 0, 0, 0, 1]], dtype=torch.uint8)
    go, gf = rand(g, N, ch, T), rand(g, N, ch, S)

    def loss(v):
        r = ref.scan(**v, flags=flags)
        return float((r["y"][0] * go).sum() + (r["final"][0] * gf).sum())

    r = ref.scan(**t, flags=flags, grad_y=go, grad_final=gf)
    for name, v in t.items():
        flat = v.reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 7)):
            step = 1e-5
            sides = []
            for sign in (1, -1):
                moved = flat.clone()
                moved[i] += sign * step
                sides.append(loss({**t, name: moved.view_as(v)}))
            slope = (sides[0] - sides[1]) / (2 * step)
            # central differences: O(step^2) and the cancellation 1e-16 / step
            assert abs(slope - float(r[name][0].reshape(-1)[i])) <= 1e-6 * (1 + abs(slope)), name


def test_a_flag_cuts_a_row_into_rows():
    g = torch.Generator().manual_seed(3)
    N, ch, S, T, cut = 1, 2, 3, 10, 4
    u, delta, A = rand(g, N, ch, T), rand(g, N, ch, T), -rand(g, ch, S).abs()
    B, C = rand(g, N, 1, S, T), rand(g, N, 1, S, T)
    flags = torch.zeros(N, T, dtype=torch.uint8)
    flags[0, cut] = 1
    whole = ref.scan(u, delta, A, B, C, flags=flags)["y"][0]
    first = ref.scan(u[..., :cut], delta[..., :cut], A, B[..., :cut], C[..., :cut])["y"][0]
    rest = ref.scan(u[..., cut:], delta[..., cut:], A, B[..., cut:], C[..., cut:])["y"][0]
    torch.testing.assert_close(whole, torch.cat([first, rest], 2), rtol=0, atol=0)
    w = rand(g, ch, 4)
    whole = ref.conv(u, w, flags=flags)["out"][0]
    parts = [ref.conv(u[..., :cut], w)["out"][0], ref.conv(u[..., cut:], w)["out"][0]]
    torch.testing.assert_close(whole, torch.cat(parts, 2), rtol=0, atol=0)
