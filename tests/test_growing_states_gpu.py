"""The selective scan where states grow: A above 0, or negative steps without
softplus.  The product of a tile's decays then passes float32's range while the
states themselves do not, from a state of 0 above all.  Against the 64-bit
reference with its bound (sequence_reference.py), forward and backward, on every
launch shape."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import sequence_reference as ref
from .test_sequence_gpu import DTYPES, NAMES, check, convention_of, episodes, gen, normal, run_scan

pytestmark = pytest.mark.gpu

# 16 lanes a row, four and two waves to four channels, or one; then four lanes and one
SHAPES = [(2, 5, 16, 150, 1), (1, 6, 3, 300, 2), (3, 1100, 4, 140, 1), (2, 3300, 5, 129, 1),
          (4, 3100, 5, 140, 1), (20, 1026, 5, 70, 1), (160, 510, 3, 13, 1)]


def compare(t, s, kw, go, gf):
    want = ref.scan(**t, state=s, grad_y=go, grad_final=gf, **kw)
    for name, (value, _) in want.items():
        assert float(value.abs().max()) < 1e37, name  # the reference stays in range
    y, final, grads = run_scan(t, s, kw["flags"], kw["lengths"], kw["convention"],
                               kw["softplus"], go, gf)
    check(y, want["y"], "y")
    check(final, want["final"], "final state")
    for name in grads._fields:
        if getattr(grads, name) is not None:
            check(getattr(grads, name), want[name], f"grad {name}")


@pytest.mark.parametrize("which", ["", "flags lengths after"], ids=lambda w: w or "plain")
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", DTYPES[:2], ids=NAMES[:2])
def test_growing(dtype, shape, which, gpu_device):
    """States that grow by up to 2^200 over a row, from inputs and gradients near
    2^-100 to 2^100.  A third of the channels see no input (states 0), and
    decaying states stand between the growing ones."""
    N, ch, S, T, G = shape
    for softplus in (True, False):
        g = gen(60 + T)
        print(f"growing {dtype} {shape} {which!r} softplus={softplus}", flush=True)
        small = 2.0 ** -100
        A = 200 / T * 0.6931 * (0.8 + 0.2 * torch.rand(ch, S, generator=g, device="cuda"))
        A[:, 1::3] *= -1
        u, go = (normal(g, N, ch, T, dtype=torch.float32, scale=small) for _ in range(2))
        u[:, ::3] = 0
        dt = 0.9 + 0.1 * torch.rand(N, ch, T, generator=g, device="cuda")
        if softplus:
            delta = torch.log(torch.expm1(dt.double())).float()
        else:
            A, delta = -A, -dt
        t = {"u": u.to(dtype), "delta": delta.to(dtype), "A": A,
             "B": normal(g, N, G, S, T, dtype=dtype), "C": normal(g, N, G, S, T, dtype=dtype),
             "z": normal(g, N, ch, T, dtype=dtype)}
        flags, lengths = episodes(g, N, T, which)
        if flags is not None:  # few starts, so that rows still grow
            flags = flags * (torch.rand(N, T, generator=g, device="cuda") < 0.05).to(torch.uint8)
        kw = dict(flags=flags, lengths=lengths, convention=convention_of(which),
                  softplus=softplus)
        compare(t, normal(g, N, ch, S, scale=small), kw, go.to(dtype),
                normal(g, N, ch, S, scale=small))
        compare(t, None, kw, go.to(dtype), None)


@pytest.mark.parametrize("flags", [False, True], ids=["plain", "flags"])
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_no_input_no_state(dtype, flags, gpu_device):
    """Steps without input leave a state of 0 at 0 whatever the growth, up to
    e^100 a step; the inputs of the last steps count."""
    g = gen(71)
    for N, ch, S, T in ((2, 5, 7, 260), (20, 1026, 5, 70), (160, 510, 3, 13)):
        delta = torch.full((N, ch, T), 100.0, device="cuda", dtype=dtype)
        delta[..., 6:] = 40.0
        delta[..., -4:] = 1.0
        u = torch.zeros(N, ch, T, device="cuda", dtype=dtype)
        u[..., -5:] = normal(g, N, ch, 5, dtype=dtype)
        u[..., -5] *= 0.01
        B, C = (normal(g, N, 1, S, T, dtype=dtype) for _ in range(2))
        t = {"u": u, "delta": delta, "A": 1.0 + torch.rand(ch, S, generator=g, device="cuda") / 8,
             "B": B, "C": C, "D": normal(g, ch)}
        f = None
        if flags:
            f = torch.zeros(N, T, dtype=torch.uint8, device="cuda")
            f[0, 3] = 1
        want = ref.scan(**t, flags=f)
        y, final, _ = rl.selective_scan(**t, flags=f, with_state=True)
        check(y, want["y"], "y")
        check(final, want["final"], "final state")


def test_small_growth_keeps_the_lane_scan(gpu_device):
    """Growth on both sides of 2^16 a tile."""
    g = gen(72)
    N, ch, S, T = 2, 40, 6, 400
    for bits in (0.02, 0.12, 0.124, 0.126, 0.13, 0.3):
        t = {"u": normal(g, N, ch, T, scale=2.0 ** -60), "B": normal(g, N, 1, S, T),
             "C": normal(g, N, 1, S, T), "delta": torch.ones(N, ch, T, device="cuda"),
             "A": torch.full((ch, S), 0.6931 * bits, device="cuda")}
        kw = dict(flags=None, lengths=None, convention=0, softplus=False)
        compare(t, normal(g, N, ch, S, scale=2.0 ** -60), kw, normal(g, N, ch, T, scale=2.0 ** -60),
                None)
