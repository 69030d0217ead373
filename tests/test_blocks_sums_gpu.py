"""The block operators' sums over sequences and steps, of terms of one sign: nothing
cancels, so the bound is the terms' own errors and the float32 roundings on one term's
way into the sum (a lane's steps, the lanes, the walkers and the waves of the last
launch), far below what one tile of one sequence contributes.  Each test checks that
it is, so that a contribution left out or added twice fails."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import blocks_reference as ref
from .sequence_reference import U, d64
from .test_blocks_launches_gpu import gated_walkers, norm_walkers
from .test_sequence_gpu import DTYPES, NAMES, gen, normal

pytestmark = pytest.mark.gpu


def last_launch(walkers):
    """Additions of a sum of walkers' parts: every 16th in turn, then the 16 waves."""
    return -(-walkers // 16) + 16


def check_sum(got, terms, errors, depth, parts, what, extra=0.0):
    """terms, errors [N, D, T] float64; parts: steps of a tile."""
    value, size = terms.sum((0, 2)), terms.abs().sum((0, 2))
    assert torch.equal(value.abs(), size), f"{what}: terms of both signs"
    bound = errors.sum((0, 2)) + (depth + extra) * U * size
    smallest = torch.stack([t.abs().sum(2) for t in terms.split(parts, 2)]).amin((0, 1))
    assert bool((bound < smallest / 2).all()), f"{what}: the bound hides a tile"
    off = (got.double().cpu() - value).abs()
    assert bool((off <= bound).all()), \
        f"{what}: off by {float((off / bound).max()):.3g} of the bound"


# lanes, waves that share a row, chunks, and a shape
GATED = [(1, 1, 1, (4200, 3, 5)), (4, 1, 1, (4200, 3, 20)), (16, 1, 1, (4200, 4, 40)),
         (16, 1, 1, (2100, 5, 128)), (64, 1, 1, (500, 9, 1024)), (64, 8, 1, (60, 20, 4096)),
         (16, 1, 2, (2, 3, 2048))]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
@pytest.mark.parametrize("case", GATED, ids=lambda c: "x".join(map(str, c[3])))
def test_gated_sums(case, dtype, gpu_device):
    lanes, waves, chunks, (N, D, T) = case
    print(f"gated sums {dtype} {N}x{D}x{T}", flush=True)
    g = gen(T)

    def about(centre, spread, *shape, dtype=torch.float32):
        return (centre + spread * torch.rand(*shape, generator=g, device="cuda")).to(dtype)

    # a state that is carried on as it is, about, so that each step's term for the decay,
    # which is (a/(1+a) - 1) times the state then, is below 0
    x = about(0.9, 0.2, N, D, T, dtype=dtype)
    gates = about(-0.1, 0.2, N, 2 * D, T, dtype=dtype)
    rate = torch.linspace(0.02, 2.0, D, device="cuda")  # of a half open gate
    decay = torch.log(torch.expm1(rate / 4))
    ib, db = about(-0.1, 0.2, D), about(-0.1, 0.2, D)
    a = torch.exp(-rate)
    state = (torch.sqrt(1 - a * a) * 0.5 / (1 - a)).expand(N, D).contiguous()
    go, gf = about(0.5, 1.0, N, D, T, dtype=dtype), about(0.5, 1.0, N, D)
    args = (x, gates[:, :D], gates[:, D:], decay)
    kw = dict(input_bias=ib, decay_bias=db, state=state)
    points = rl.gated_recurrence(*args, with_checkpoints=True, **kw)[2]
    tiles = -(-T // (8 * lanes))
    assert points.numel() == N * D * tiles
    grads = rl.gated_recurrence_backward(go, *args, points, grad_state=gf, **kw)
    want = ref.gated(*args, grad_out=go, grad_final=gf, **kw)
    if chunks > 1:
        walkers, serial = 4096, 8 * tiles
    else:
        walkers = gated_walkers(N, D, T, dtype)
        serial = 8 * -(-tiles // waves) * -(-N * waves // walkers)
    depth = serial + 6 + last_launch(walkers)
    gi, gi_e = want["input_gate"]
    gr, gr_e = want["decay_gate"]
    check_sum(grads.input_bias, gi, gi_e, depth, 8 * lanes, "input bias")
    check_sum(grads.decay_bias, gr, gr_e, depth, 8 * lanes, "decay bias")
    # e = grad_decay_gate / (1 - r), and its sum times sigmoid(decay) / softplus(decay)
    kept = 1 - torch.sigmoid(d64(gates[:, D:]) + d64(db)[:, None])
    ratio = torch.sigmoid(d64(decay)) / ref.softplus(d64(decay))
    check_sum(grads.decay.cpu() / ratio, gr / kept, gr_e / kept, depth, 8 * lanes, "decay", 24)


NORM = [(600, 520, 7), (600, 100, 9), (600, 300, 9), (9, 530, 3648), (80, 2100, 64), (700, 33, 64)]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
@pytest.mark.parametrize("shape", NORM, ids=lambda s: "x".join(map(str, s)))
def test_norm_sums(shape, dtype, gpu_device):
    N, D, T = shape
    print(f"norm sums {dtype} {N}x{D}x{T}", flush=True)
    g = gen(T + D)
    x = (0.5 + torch.rand(N, D, T, generator=g, device="cuda")).to(dtype)
    go = (0.5 + torch.rand(N, D, T, generator=g, device="cuda")).to(dtype)
    w = 1 + normal(g, D, scale=0.3)
    grads = rl.rms_norm_backward(go, x, w)
    s = d64(x)
    xh = s / torch.sqrt((s * s).mean(1, keepdim=True) + ref.EPS)
    terms = d64(go) * xh
    n = D / 32 + 16  # as the reference counts a sum over channels
    vec = 16 // dtype.itemsize
    walkers = norm_walkers(x)
    # a thread's steps of its tiles, at least 16 bytes wide, and up to 8 lanes
    serial = vec * -(-N * -(-T // vec) // walkers)
    check_sum(grads.weight, terms, terms * (n / 2 + 4 + 2) * U, serial + 3 + last_launch(walkers),
              64, "weight")


@pytest.mark.parametrize("N,D", [(2100, 300), (600, 5000), (5000, 40)])
def test_norm_sums_of_dense_rows(N, D, gpu_device):
    for dtype in DTYPES:
        g = gen(D)
        x = (0.5 + torch.rand(N, D, generator=g, device="cuda")).to(dtype)
        go = (0.5 + torch.rand(N, D, generator=g, device="cuda")).to(dtype)
        grads = rl.rms_norm_backward(go, x, torch.ones(D, device="cuda"))
        s = d64(x)
        terms = (d64(go) * s / torch.sqrt((s * s).mean(1, keepdim=True) + ref.EPS))[:, :, None]
        walkers = norm_walkers(x[:, :, None])
        check_sum(grads.weight, terms, terms * ((D / 32 + 16) / 2 + 6) * U,
                  -(-N // walkers) + last_launch(walkers), 1, "weight")
