"""Seeded random calls of the sequence operators: shapes on every launch shape,
storage types, flag densities, conventions, lengths, optional inputs and views
at odd offsets, each against the 64-bit reference within its bound."""
import random

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import sequence_reference as ref
from .test_sequence_gpu import DTYPES, check, gen, normal

pytestmark = pytest.mark.gpu


def view(r, g, N, D, T, dtype, scale=1.0):
    """[N, D, T] inside a larger array, at an odd offset in every dimension."""
    d, t = r.choice([0, 0, 1, 3]), r.choice([0, 0, 1, 2, 5, 8])
    wide = normal(g, N, D + d, T + t + r.choice([0, 0, 1, 4, 7]), dtype=dtype, scale=scale)
    return wide[:, d:, t:t + T]


def boundaries(r, g, N, T):
    flags = lengths = None
    if r.random() < 0.6:
        flags = (torch.rand(N, T, generator=g, device="cuda") < r.choice([0.01, 0.1, 0.6]))
        flags = flags if r.random() < 0.5 else flags.to(torch.uint8) * 7
    if r.random() < 0.4:
        lengths = torch.randint(0, T + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    return dict(flags=flags, lengths=lengths,
                convention=r.choice([rl.RESET_ON_START, rl.RESET_AFTER_DONE]))


def length(r):
    return r.choice([r.randint(1, 9), r.randint(1, 40), r.randint(30, 140), r.randint(120, 700)])


def conv_case(seed):
    r, g = random.Random(seed), gen(seed)
    dtype, T, W = r.choice(DTYPES), length(r), r.randint(2, 4)
    rows = max(1, min(r.choice([3, 40, 3000]), 400_000 // T))
    D = r.randint(1, max(1, min(rows, 300)))
    N = max(1, rows // D)
    print(f"conv seed {seed}: {dtype} {N}x{D}x{T} W={W}", flush=True)
    x, go = view(r, g, N, D, T, dtype), view(r, g, N, D, T, dtype)
    w = normal(g, D, W, scale=0.6)
    b = normal(g, D) if r.random() < 0.7 else None
    s = normal(g, N, D, W - 1, dtype=dtype) if r.random() < 0.5 else None
    gf = normal(g, N, D, W - 1, dtype=dtype) if r.random() < 0.5 else None
    kw = dict(boundaries(r, g, N, T), state=s, silu=r.random() < 0.8)
    want = ref.conv(x, w, b, grad_out=go, grad_final=gf, **kw)
    out, final = rl.causal_conv(x, w, b, with_state=True, **kw)
    check(out, want["out"], "out")
    check(final, want["final"], "final state")
    grads = rl.causal_conv_backward(go, x, w, b, grad_state=gf, **kw)
    for name in grads._fields:
        if getattr(grads, name) is not None:
            check(getattr(grads, name), want[name], f"grad {name}")


def scan_case(seed):
    r, g = random.Random(seed), gen(seed)
    dtype, T, G = r.choice(DTYPES), length(r), r.choice([1, 1, 2, 3])
    S = r.choice([r.randint(1, 8), r.randint(1, 20), 16, r.randint(17, 128)])
    # few rows, or enough for a wave alone, for four lanes a row, for one
    rows = max(1, min(r.choice([4, 60, 9000, 30_000, 100_000]), 5_000_000 // (T * S)))
    D = G * r.randint(1, max(1, min(rows, 700) // G))
    N = max(1, rows // D)
    print(f"scan seed {seed}: {dtype} {N}x{D}x{T} S={S} G={G}", flush=True)
    softplus = r.random() < 0.7
    t = dict(u=view(r, g, N, D, T, dtype), delta=view(r, g, N, D, T, dtype),
             A=-(0.05 + 2 * torch.rand(D, S, generator=g, device="cuda")),
             B=view(r, g, N * G, S, T, dtype).unflatten(0, (N, G)),
             C=view(r, g, N * G, S, T, dtype).unflatten(0, (N, G)))
    if not softplus:
        t["delta"] = t["delta"].abs() * 0.1
    if r.random() < 0.6:
        t["D"] = normal(g, D)
    if r.random() < 0.6:
        t["z"] = view(r, g, N, D, T, dtype)
    if softplus and r.random() < 0.6:
        t["delta_bias"] = normal(g, D) - 2
    s = normal(g, N, D, S) if r.random() < 0.5 else None
    gf = normal(g, N, D, S) if r.random() < 0.5 else None
    go = view(r, g, N, D, T, dtype)
    kw = dict(boundaries(r, g, N, T), state=s, softplus=softplus)
    want = ref.scan(**t, grad_y=go, grad_final=gf, **kw)
    y, final, points = rl.selective_scan(**t, with_state=True, with_checkpoints=True, **kw)
    check(y, want["y"], "y")
    check(final, want["final"], "final state")
    grads = rl.selective_scan_backward(go, **t, checkpoints=points, grad_state=gf, **kw)
    for name in grads._fields:
        if getattr(grads, name) is not None:
            check(getattr(grads, name), want[name], f"grad {name}")


@pytest.mark.parametrize("seed", range(20))
def test_random_conv(seed, gpu_device):
    conv_case(seed)


@pytest.mark.parametrize("seed", range(1000, 1032))
def test_random_scan(seed, gpu_device):
    scan_case(seed)
