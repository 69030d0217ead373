"""Seeded random calls of the block and beam operators over every launch shape, against
the 64-bit references: sizes, types, strides, episodes under both conventions, lengths,
states, biases, masked tokens and beams that are finished or not in use."""
import random

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import test_beams_gpu as beams
from .test_gated_gpu import inputs, run_all
from .test_norm_gpu import check_all
from .test_sequence_gpu import DTYPES, episodes, gen, normal

pytestmark = pytest.mark.gpu


def log_int(r, lo, hi):
    return int(round(lo * (hi / lo) ** r.random()))


@pytest.mark.parametrize("seed", range(24))
def test_gated(seed, gpu_device):
    r = random.Random(seed)
    g = gen(seed)
    # rows of every kind: short, many, few and long, very few and very long
    T = log_int(r, 1, 6000)
    rows = log_int(r, 1, max(1, min(9000, 600_000 // T)))
    D = log_int(r, 1, rows)
    N = max(1, rows // D)
    dtype, which = r.choice(DTYPES), r.choice(["", "flags", "flags after", "lengths",
                                               "flags lengths", "flags lengths after"])
    full = r.random() < 0.6
    scale = r.choice([8.0, 8.0, 1.0, 30.0])
    print(f"gated {dtype} {which!r} {N}x{D}x{T} full={full} scale={scale}", flush=True)
    a = inputs(g, N, D, T, dtype, full)
    skew = r.randint(0, 3)  # rows that begin anywhere
    if skew:
        wide = normal(g, N, D + 1, T + skew, dtype=dtype)
        a["x"] = wide[:, 1:, skew:]
    if r.random() < 0.5:
        a["decay"] = torch.full_like(a["decay"], -5.0)  # slow throughout
    go = normal(g, N, D, T, dtype=dtype)
    gf = normal(g, N, D) if r.random() < 0.5 else None
    flags, lengths = episodes(g, N, T, which)
    run_all(a, which, flags, lengths, go, gf, scale=scale)


@pytest.mark.parametrize("seed", range(24))
def test_norm(seed, gpu_device):
    r = random.Random(100 + seed)
    g = gen(seed)
    D = log_int(r, 1, 9000)
    T = 1 if r.random() < 0.3 else log_int(r, 1, 700)
    N = log_int(r, 1, max(1, min(3000, 3_000_000 // (D * T))))
    dtype = r.choice(DTYPES)
    skew = r.randint(0, 3)
    which = r.choice(["", "", "lengths"])
    print(f"norm {dtype} {which!r} {N}x{D}x{T} skew={skew}", flush=True)

    def array(scale=1.0):
        return normal(g, N, D + 1, T + skew, dtype=dtype, scale=scale)[:, 1:, skew:]

    w = normal(g, D) if r.random() < 0.7 else None
    res = array(2.0) if r.random() < 0.6 else None
    gs = array() if r.random() < 0.6 else None
    lengths = episodes(g, N, T, which)[1]
    x, go = array(), array()
    if T == 1 and r.random() < 0.5:  # dense rows of channels
        x, go, res, gs = (None if t is None else t[:, :, 0].contiguous() for t in (x, go, res, gs))
    check_all(x, w, res, go, gs, lengths)


@pytest.mark.parametrize("seed", range(24))
def test_beams(seed, gpu_device):
    r = random.Random(200 + seed)
    g = gen(seed)
    K = r.choice([1, 2, 3, 5, 8, 17, 64])
    V = log_int(r, 1, 30000)
    N = log_int(r, 1, max(1, min(60, 1_500_000 // (K * V))))
    picks = min(64, K * V, r.choice([1, K, 2 * K, 64]))
    dtype = r.choice(DTYPES)
    print(f"beams {dtype} {N}x{K}x{V} picks {picks}", flush=True)
    logits = normal(g, N, K + 1, V + 3, dtype=dtype, scale=r.choice([0.1, 1.0, 5.0]))
    logits = logits[:, :K, r.randint(0, 3):][:, :, :V]
    if r.random() < 0.4:
        mask = torch.rand(N, K, V, generator=g, device="cuda") < r.choice([0.3, 0.9, 0.999])
        logits = logits.masked_fill(mask, -float("inf"))
    scores = -10 * torch.rand(N, K, generator=g, device="cuda")
    if r.random() < 0.4:
        scores[torch.rand(N, K, generator=g, device="cuda") < 0.4] = -float("inf")
    kw = {}
    if r.random() < 0.5:
        kw = dict(finished=torch.rand(N, K, generator=g, device="cuda") < 0.3,
                  pad_token=r.randrange(V))
    choice = beams.check(logits, scores, picks, **kw)
    if picks == K:
        places = N * K + r.randint(0, 9)
        pools = beams.pools_of(g, places)
        slots = torch.randperm(places, generator=g, device="cuda")[:N * K].int().view(N, K)
        want, new = beams.reordered(pools, slots, choice.parents)
        assert torch.equal(rl.beam_reorder(pools, slots, choice.parents).cpu(), new)
        assert all(torch.equal(p, w) for p, w in zip(pools, want))
