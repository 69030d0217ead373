"""The block operators where a wave or workgroup walks several sequences or tiles, and in
the launch shapes that other tests' sizes do not reach, against the 64-bit references.
Each test states, from the sizes that the library answers, that it reaches its shape."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from linear_recurrence_scan_row_amd import blocks
from linear_recurrence_scan_row_amd.rlca import REAL_DTYPES, lib
from . import blocks_reference as ref
from .test_gated_gpu import inputs, run_all
from .test_norm_gpu import check_all
from .test_sequence_gpu import DTYPES, NAMES, WHICH, check, convention_of, episodes, gen, normal

pytestmark = pytest.mark.gpu


def gated_walkers(N, D, T, dtype):
    """How many workers share a channel group's sequences in the backward call, from its
    workspace: three floats a channel for each wave (no chunks at these sizes)."""
    call = blocks.GatedCall(num_seqs=N, channels=D, T=T, dtype=REAL_DTYPES[dtype], scale=8.0)
    n = lib().rlca_gated_recurrence_backward_workspace_size(bytes(call))
    assert n % (12 * D) == 0
    return n // (12 * D)


def norm_walkers(x):
    """The same for the norm: one float a channel for each."""
    N, D, T = x.shape
    call = blocks.NormCall(num_seqs=N, channels=D, T=T, dtype=REAL_DTYPES[x.dtype], eps=1e-6,
                           x=x.data_ptr(), x_stride_seq=x.stride(0), x_stride_channel=x.stride(1),
                           grad_out=x.data_ptr(), grad_stride_seq=x.stride(0),
                           grad_stride_channel=x.stride(1))
    return lib().rlca_rms_norm_backward_workspace_size(bytes(call)) // (4 * D)


# lanes a row, waves that share it, and a shape in which each walks several sequences
WALKS = [(1, 1, (4200, 3, 5)), (4, 1, (4200, 3, 20)), (16, 1, (4200, 4, 40)),
         (16, 1, (2100, 5, 150)), (64, 1, (1400, 3, 1000)), (64, 8, (600, 2, 2100))]


@pytest.mark.parametrize("which", WHICH, ids=lambda w: w.replace(" ", "_") or "plain")
@pytest.mark.parametrize("walk", WALKS, ids=lambda w: f"{w[0]}x{w[1]}-{'x'.join(map(str, w[2]))}")
def test_gated_workers_walk_sequences(walk, which, gpu_device):
    lanes, waves, (N, D, T) = walk
    for dtype in DTYPES if T < 200 else (torch.bfloat16,):
        print(f"gated {dtype} {which!r} {N}x{D}x{T}", flush=True)
        assert gated_walkers(N, D, T, dtype) // waves < N
        g = gen(T)
        a = inputs(g, N, D, T, dtype, True)
        tiles = -(-T // (8 * lanes))
        points = rl.gated_recurrence(a["x"], a["input_gate"], a["decay_gate"], a["decay"],
                                     with_checkpoints=True)[2]
        assert points.numel() == N * D * tiles
        flags, lengths = episodes(g, N, T, which)
        run_all(a, which, flags, lengths, normal(g, N, D, T, dtype=dtype), normal(g, N, D))


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
@pytest.mark.parametrize("slots", [False, True], ids=["dense", "slots"])
def test_gated_step_walks_sequences(slots, dtype, gpu_device):
    """More sequences than 2048 workgroups of 256 channels hold."""
    for N, D in ((2100, 64), (4097, 3), (700, 1030), (1025, 500), (300, 2600)):
        assert N > -(-2048 // -(-D // 256))
        print(f"gated step {dtype} {N}x{D} slots={slots}", flush=True)
        g = gen(N)
        places = N + 5
        a = inputs(g, N, D, 1, dtype, True)
        x, ig, dg = (a[k][:, :, 0] for k in ("x", "input_gate", "decay_gate"))
        x = x.contiguous()
        ig, dg = torch.cat([ig, dg], 1).split(D, 1)
        state = normal(g, places, D)
        before = state.clone()
        starts = (torch.rand(N, generator=g, device="cuda") < 0.3).to(torch.uint8)
        at = torch.randperm(places, generator=g, device="cuda")[:N] if slots \
            else torch.arange(N, device="cuda")
        seat = at.int()
        if slots:
            seat[::7] = -1  # empty seats
        out = rl.gated_step(x, ig, dg, a["decay"], state, a["input_bias"], a["decay_bias"],
                            slots=seat if slots else None, flags=starts)
        want = ref.gated(x[:, :, None], ig[:, :, None], dg[:, :, None], a["decay"],
                         a["input_bias"], a["decay_bias"], state=before[at],
                         flags=starts[:, None])
        used = seat.cpu() >= 0
        check(out[used.cuda()][:, :, None], [w[used] for w in want["out"]], "out")
        check(state[at[used.cuda()]], [w[used] for w in want["final"]], "state")
        assert not out[~used.cuda()].any()
        others = torch.ones(places, dtype=torch.bool, device="cuda")
        others[at[used.cuda()]] = False
        assert torch.equal(state[others], before[others])


# (sequences, channels, steps by type): tiles of 4 x 16 bytes of a channel's steps, for few
# whole rows and for many channels; and those and wider ones that walk in the backward call
ROWS = [((4, 600), {4: 512, 2: 1024}, False), ((4, 601), {4: 515, 2: 1027}, False),
        ((5, 530), {4: 832, 2: 1664}, False), ((5, 2100), {4: 230, 2: 460}, False),
        ((600, 2100), {4: 5, 2: 5}, True), ((600, 520), {4: 7, 2: 7}, True),
        ((9, 530), {4: 1900, 2: 3700}, True), ((600, 300), {4: 9, 2: 9}, True),
        ((600, 100), {4: 9, 2: 9}, True)]


@pytest.mark.parametrize("which", ["", "lengths"], ids=["plain", "lengths"])
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
@pytest.mark.parametrize("shape", ROWS, ids=lambda s: "x".join(map(str, s[0])))
def test_norm_of_rows(shape, dtype, which, gpu_device):
    (N, D), steps, walks = shape
    T = steps[dtype.itemsize]
    print(f"norm {dtype} {which!r} {N}x{D}x{T}", flush=True)
    g = gen(N + T)
    x, go = normal(g, N, D, T, dtype=dtype), normal(g, N, D, T, dtype=dtype)
    assert (norm_walkers(x) == 512) == walks
    w = 1 + normal(g, D, scale=0.3)
    res, gs = normal(g, N, D, T, dtype=dtype, scale=2.0), normal(g, N, D, T, dtype=dtype)
    check_all(x, w, res, go, gs, episodes(g, N, T, which)[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_norm_of_dense_rows_that_walk(dtype, gpu_device):
    """Rows of channels: a wave and a workgroup walk several, beyond what registers hold too."""
    for N, D in ((2100, 300), (5000, 40), (600, 5000), (600, 9001)):
        print(f"norm {dtype} {N}x{D}", flush=True)
        g = gen(D)
        x, go, res, gs = (normal(g, N, D, dtype=dtype) for _ in range(4))
        assert norm_walkers(x[:, :, None]) in (512, 2048) and norm_walkers(x[:, :, None]) < N
        check_all(x, normal(g, D), res, go, gs, None)
