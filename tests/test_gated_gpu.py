"""The gated recurrence's kernels against the 64-bit reference, each output within
the bound that the reference carries for float32 arithmetic plus one rounding to
its type (blocks_reference.py): storage types, row lengths on both sides of a
lane's block, of a tile and of a chunk, strides, episodes under both conventions,
lengths from 0, slow and fast decays, and what may not pass an episode's start or
a row's end."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import blocks_reference as ref
from .test_sequence_gpu import DTYPES, NAMES, WHICH, check, convention_of, episodes, gen, normal

pytestmark = pytest.mark.gpu


def decays(g, D):
    """softplus(decay) from 1e-4 to a few, both sides of the polynomial's range."""
    if D == 1:
        return torch.full((1,), -3.0, device="cuda")
    return torch.linspace(-9, 2, D, device="cuda")[torch.randperm(D, generator=g, device="cuda")]


def inputs(g, N, D, T, dtype, full, scale=1.0):
    gates = normal(g, N, 2 * D, T, dtype=dtype, scale=2.0)
    return dict(x=normal(g, N, D, T, dtype=dtype, scale=scale), input_gate=gates[:, :D],
                decay_gate=gates[:, D:], decay=decays(g, D),
                input_bias=normal(g, D) if full else None,
                decay_bias=normal(g, D) if full else None,
                state=normal(g, N, D) if full else None)


def run_all(a, which, flags, lengths, go, gf, scale=8.0):
    args = (a["x"], a["input_gate"], a["decay_gate"], a["decay"])
    kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], scale=scale,
              state=a["state"], flags=flags, convention=convention_of(which), lengths=lengths)
    want = ref.gated(*args, grad_out=go, grad_final=gf, **kw)
    out, final, points = rl.gated_recurrence(*args, with_state=True, with_checkpoints=True, **kw)
    check(out, want["out"], "out")
    check(final, want["final"], "final")
    grads = rl.gated_recurrence_backward(go, *args, points, grad_state=gf, **kw)
    for name in rl.GatedGrads._fields:
        got = getattr(grads, name)
        if got is not None:
            check(got, want[name], f"grad {name}")
        else:
            assert a[name] is None
    return out, final, grads


# rows of 1, 4, 16 and 64 lanes, of several tiles, rows that a workgroup shares, and of
# several chunks
SHAPES = [(5, 3, 1), (5, 70, 2), (6, 65, 7), (5, 5, 8), (5, 17, 9), (5, 3, 31), (5, 18, 32),
          (5, 3, 33), (5, 5, 127), (5, 4, 128), (5, 3, 130), (5, 6, 515), (3, 5, 1031),
          (2, 3, 2051), (1, 2, 4100), (2100, 2, 300), (2100, 3, 500), (5, 30, 1100), (2, 60, 2600),
          (1, 100, 8200)]


@pytest.mark.parametrize("which", WHICH, ids=lambda w: w.replace(" ", "_") or "plain")
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_gated(dtype, which, gpu_device):
    for N, D, T in SHAPES:
        for full in (True, False):
            g = gen(100 + T)
            print(f"gated {dtype} {which!r} {N}x{D}x{T} full={full}", flush=True)
            a = inputs(g, N, D, T, dtype, full)
            go = normal(g, N, D, T, dtype=dtype)
            gf = normal(g, N, D) if full else None
            flags, lengths = episodes(g, N, T, which)
            run_all(a, which, flags, lengths, go, gf)


def test_gated_scales(gpu_device):
    """Rates from where nothing decays to where nothing is kept."""
    g = gen(5)
    a = inputs(g, 3, 40, 77, torch.float32, True)
    go, gf = normal(g, 3, 40, 77), normal(g, 3, 40)
    for scale in (1e-6, 0.01, 1.0, 40.0, 1e4):
        print(f"scale {scale}", flush=True)
        run_all(a, "", None, None, go, gf, scale=scale)


def test_gated_empty(gpu_device):
    g = gen(6)
    for N, D, T in ((0, 3, 9), (3, 0, 9), (3, 5, 0), (0, 3, 0)):
        a = inputs(g, N, D, T, torch.float32, True)
        args = (a["x"], a["input_gate"], a["decay_gate"], a["decay"])
        kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], state=a["state"])
        out, final, points = rl.gated_recurrence(*args, with_state=True, with_checkpoints=True,
                                                 **kw)
        gf = normal(g, N, D)
        grads = rl.gated_recurrence_backward(normal(g, N, D, T), *args, points, grad_state=gf,
                                             **kw)
        assert out.shape == (N, D, T) and grads.x.shape == (N, D, T)
        if T == 0:
            assert torch.equal(final, a["state"]) and torch.equal(grads.state, gf)
        assert not grads.decay.any() and not grads.input_bias.any() and not grads.decay_bias.any()


def test_gated_rows_continue(gpu_device):
    """A row in two calls, the state handed on, is the row in one."""
    g = gen(1)
    a = inputs(g, 3, 5, 300, torch.float32, True)
    args = (a["input_gate"], a["decay_gate"])
    kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], with_state=True)
    whole, final, _ = rl.gated_recurrence(a["x"], *args, a["decay"], state=a["state"], **kw)
    for cut in (1, 8, 31, 128, 299):
        first, s, _ = rl.gated_recurrence(a["x"][..., :cut], *(t[..., :cut] for t in args),
                                          a["decay"], state=a["state"], **kw)
        rest, f, _ = rl.gated_recurrence(a["x"][..., cut:], *(t[..., cut:] for t in args),
                                         a["decay"], state=s, **kw)
        torch.testing.assert_close(torch.cat([first, rest], 2), whole, rtol=2e-5, atol=2e-5)
        torch.testing.assert_close(f, final, rtol=2e-5, atol=2e-5)


def test_gated_strided_views(gpu_device):
    g = gen(2)
    for dtype in DTYPES:
        wide = normal(g, 4, 12, 99, dtype=dtype)
        decay = decays(g, 4)
        for x, ig, dg in ((wide[:, :4, 1:], wide[:, 4:8, :98], wide[:, ::3, 1:]),
                          (wide[:1, :4].expand(4, 4, 99), wide[:, :1].expand(4, 4, 99),
                           wide[::1, 8:]),):
            kw = dict(with_state=True, with_checkpoints=True)
            out, final, c = rl.gated_recurrence(x, ig, dg, decay, **kw)
            dense = [t.contiguous() for t in (x, ig, dg)]
            out1, final1, c1 = rl.gated_recurrence(*dense, decay, **kw)
            assert torch.equal(out, out1) and torch.equal(final, final1)
            go = normal(g, 4, 9, x.shape[2], dtype=dtype)[:, 3:7]
            p = rl.gated_recurrence_backward(go, x, ig, dg, decay, c)
            q = rl.gated_recurrence_backward(go.contiguous(), *dense, decay, c1)
            for u, v in zip(p, q):
                assert (u is None and v is None) or torch.equal(u, v)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_gated_step(dtype, gpu_device):
    # the last two: four channels a thread, workgroups that walk several sequences
    for N, D, slots in ((1, 1, False), (3, 7, False), (5, 64, True), (2, 300, True),
                        (1, 2048, False), (300, 1003, True), (520, 600, False)):
        g = gen(10 + D)
        print(f"gated step {dtype} {N}x{D} slots={slots}", flush=True)
        places = N + 3
        a = inputs(g, N, D, 1, dtype, True)
        state = normal(g, places, D)
        before = state.clone()
        starts = (torch.rand(N, generator=g, device="cuda") < 0.4).to(torch.uint8)
        at = torch.randperm(places, generator=g, device="cuda")[:N] if slots \
            else torch.arange(N, device="cuda")
        wide = normal(g, N, 3 * D + 5, dtype=dtype)
        x, ig, dg = wide[:, 2:D + 2], wide[:, D + 3:2 * D + 3], wide[:, 2 * D + 5:]
        out = rl.gated_step(x, ig, dg, a["decay"], state, a["input_bias"], a["decay_bias"],
                            slots=at.int() if slots else None, flags=starts)
        want = ref.gated(x[:, :, None], ig[:, :, None], dg[:, :, None], a["decay"],
                         a["input_bias"], a["decay_bias"], state=before[at],
                         flags=starts[:, None])
        check(out[:, :, None], want["out"], "out")
        check(state[at], want["final"], "state")
        others = torch.ones(places, dtype=torch.bool, device="cuda")
        others[at] = False
        assert torch.equal(state[others], before[others])


def test_gated_step_empty_seats(gpu_device):
    g = gen(11)
    a = inputs(g, 4, 9, 1, torch.float32, True)
    state = normal(g, 3, 9)
    before = state.clone()
    slots = torch.tensor([-1, 2, 3, 0], device="cuda", dtype=torch.int32)
    x, ig, dg = (a[k][:, :, 0].contiguous() for k in ("x", "input_gate", "decay_gate"))
    out = rl.gated_step(x, ig, dg, a["decay"], state, slots=slots)
    assert not out[0].any() and not out[2].any() and out[1].any() and out[3].any()
    assert torch.equal(state[1], before[1]) and not torch.equal(state[2], before[2])


def test_gated_nothing_passes_a_start_or_an_end(gpu_device):
    """NaN and infinity before an episode's start and past a row's length."""
    g = gen(12)
    for T in (7, 30, 130, 2051):
        N, D = 2, 5
        a = inputs(g, N, D, T, torch.float32, True)
        go, gf = normal(g, N, D, T), normal(g, N, D)
        cut, end = T // 2, T - 2
        flags = torch.zeros(N, T, device="cuda", dtype=torch.uint8)
        flags[:, cut] = 1
        lengths = torch.full((N,), end, device="cuda", dtype=torch.int32)
        kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], flags=flags,
                  lengths=lengths)

        def run(x, ig, dg, go, state):
            args = (x.clone(), ig.clone(), dg.clone(), a["decay"])
            out, final, c = rl.gated_recurrence(*args, state=state, with_state=True,
                                                with_checkpoints=True, **kw)
            return out, final, rl.gated_recurrence_backward(go, *args, c, state=state,
                                                            grad_state=gf, **kw)

        x, ig, dg = a["x"], a["input_gate"].clone(), a["decay_gate"].clone()
        want = run(x, ig, dg, go, a["state"])
        for bad in (float("nan"), float("inf"), -float("inf")):
            # before the start: nothing after it changes
            x1, s1, go1 = x.clone(), a["state"].clone(), go.clone()
            x1[:, :, :cut] = bad
            s1[:] = bad
            got = run(x1, ig, dg, go, s1)
            assert torch.equal(got[0][:, :, cut:], want[0][:, :, cut:])
            assert torch.equal(got[1], want[1])
            for name in ("x", "input_gate", "decay_gate"):
                assert torch.equal(getattr(got[2], name)[:, :, cut:],
                                   getattr(want[2], name)[:, :, cut:])
            # a gradient after the start reaches nothing before it
            go1[:, :, cut:end] = bad
            got = run(x, ig, dg, go1, a["state"])
            assert torch.equal(got[2].state, want[2].state)
            for name in ("x", "input_gate", "decay_gate"):
                assert torch.equal(getattr(got[2], name)[:, :, :cut],
                                   getattr(want[2], name)[:, :, :cut])
            # past the end: nothing is used
            x2, ig2, dg2, go2 = x.clone(), ig.clone(), dg.clone(), go.clone()
            for t in (x2, ig2, dg2, go2):
                t[:, :, end:] = bad
            got = run(x2, ig2, dg2, go2, a["state"])
            for p, q in zip((got[0], got[1], *got[2]), (want[0], want[1], *want[2])):
                assert torch.equal(p, q)


def test_gated_masked_gates(gpu_device):
    """Gates masked by the type's lowest value or an infinity: a closed input gate lets
    nothing in, a closed decay gate keeps the state, open ones do as the formula says."""
    for dtype in DTYPES:
        low = torch.finfo(dtype).min
        for closed in (low, -float("inf")):
            g = gen(13)
            a = inputs(g, 2, 6, 140, dtype, False)
            state = normal(g, 2, 6)
            ig = torch.full((2, 6, 140), closed, device="cuda", dtype=dtype)
            out, final, c = rl.gated_recurrence(a["x"], a["input_gate"], ig, a["decay"],
                                                state=state, with_state=True,
                                                with_checkpoints=True)
            assert torch.equal(final, state)  # L = 0: a = 1 and the input's weight 0
            grads = rl.gated_recurrence_backward(torch.ones_like(out), a["x"], a["input_gate"],
                                                 ig, a["decay"], c, state=state)
            assert torch.equal(grads.state, torch.full_like(state, 140.0))
            for t in (grads.x, grads.decay_gate, grads.decay):
                assert torch.isfinite(t).all() and not t.any()
            out, final, _ = rl.gated_recurrence(a["x"], ig, a["decay_gate"], a["decay"],
                                                with_state=True)
            assert not out.any() and not final.any()
        top = torch.full((2, 6, 140), -low, device="cuda", dtype=dtype)
        want = ref.gated(a["x"], top, a["decay_gate"], a["decay"])
        check(rl.gated_recurrence(a["x"], top, a["decay_gate"], a["decay"])[0], want["out"], "open")


def test_gated_gradients_against_differences(gpu_device):
    g = gen(14)
    N, D, T = 2, 3, 21
    a = inputs(g, N, D, T, torch.float32, True)
    go, gf = normal(g, N, D, T), normal(g, N, D)
    names = ("x", "input_gate", "decay_gate", "decay", "input_bias", "decay_bias", "state")

    def loss(v):
        w = ref.gated(v["x"], v["input_gate"], v["decay_gate"], v["decay"], v["input_bias"],
                      v["decay_bias"], state=v["state"])
        return float((w["out"][0] * go.cpu()).sum() + (w["final"][0] * gf.cpu()).sum())

    args = (a["x"], a["input_gate"], a["decay_gate"], a["decay"])
    kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], state=a["state"])
    c = rl.gated_recurrence(*args, with_checkpoints=True, **kw)[2]
    grads = rl.gated_recurrence_backward(go, *args, c, grad_state=gf, **kw)
    for name in names:
        v = {k: t.cpu().double().clone() for k, t in a.items()}
        step = normal(g, *a[name].shape).cpu().double()
        up, down = dict(v), dict(v)
        up[name], down[name] = v[name] + 1e-5 * step, v[name] - 1e-5 * step
        slope = (loss(up) - loss(down)) / 2e-5
        got = float((getattr(grads, name).cpu().double() * step).sum())
        # central differences: 1e-10 of third derivatives, 1e-16 / 1e-5 of rounding
        scale = float((getattr(grads, name).cpu().double().abs() * step.abs()).sum())
        assert abs(got - slope) <= 1e-5 * (scale + 1), name


def test_gated_captured_and_streams(gpu_device):
    """Calls in a captured graph, replayed with the eager ones between, and on another
    stream."""
    g = gen(15)
    a = inputs(g, 2, 70, 2051, torch.bfloat16, True)
    go = normal(g, 2, 70, 2051, dtype=torch.bfloat16)
    args = (a["x"], a["input_gate"], a["decay_gate"], a["decay"])
    kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], state=a["state"])

    def both():
        out, f, c = rl.gated_recurrence(*args, with_state=True, with_checkpoints=True, **kw)
        return out, f, *rl.gated_recurrence_backward(go, *args, c, **kw)

    want = [t.clone() for t in both()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = both()
    torch.cuda.synchronize()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        eager = both()
        torch.cuda.synchronize()
        for p, q, w in zip(got, eager, want):
            assert torch.equal(p, w) and torch.equal(q, w)
