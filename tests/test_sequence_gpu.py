"""The sequence operators' kernels against the 64-bit reference, each output
within the bound that the reference carries for float32 arithmetic plus one
rounding to its type (sequence_reference.py): storage types, row lengths on
both sides of a lane's block and of a tile, state and tap counts, groups,
strides, episodes under both conventions, lengths from 0, and what may not
pass an episode's start or a row's end."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import sequence_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = ["f32", "bf16", "f16"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def check(got, want, what):
    value, bound = want
    got64 = got.detach().cpu().double()
    assert got64.shape == value.shape, f"{what}: shape {tuple(got64.shape)}"
    tol = ref.tolerance(value, bound, got.dtype)
    off = (got64 - value).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} values off, the first at {i}: "
                    f"{float(got64[i])!r}, expected {float(value[i])!r} within {float(tol[i]):.3e}")


def episodes(g, N, T, which):
    flags = lengths = None
    if "flags" in which:
        flags = (torch.rand(N, T, generator=g, device="cuda") < 0.1).to(torch.uint8) * 3
        if T > 0 and N > 1:
            flags[1, T - 1] = 1
            flags[0, 0] = 1
    if "lengths" in which:
        lengths = torch.randint(0, T + 1, (N,), generator=g, device="cuda").to(torch.int32)
        lengths[0] = 0
        if N > 2:
            lengths[1], lengths[2] = T, min(T, 1)
        if N > 4:
            lengths[3], lengths[4] = -5, T + 9  # taken as 0 and T
    return flags, lengths


WHICH = ["", "flags", "flags after", "lengths", "flags lengths after"]


def convention_of(which):
    return rl.RESET_AFTER_DONE if "after" in which else rl.RESET_ON_START


# ------------------------------------------------------------- the convolution
CONV_SHAPES = [(5, 3, 1), (5, 3, 2), (5, 7, 3), (6, 2, 7), (5, 5, 8), (5, 3, 9), (5, 2, 17),
               (5, 3, 64), (5, 2, 130), (5, 1, 515), (5, 2, 2051)]


@pytest.mark.parametrize("which", WHICH, ids=lambda w: w.replace(" ", "_") or "plain")
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_conv(dtype, W, which, gpu_device):
    for N, D, T in CONV_SHAPES:
        for full in (True, False):
            g = gen(100 + T)
            print(f"conv {dtype} W={W} {which!r} {N}x{D}x{T} full={full}", flush=True)
            x, go = normal(g, N, D, T, dtype=dtype), normal(g, N, D, T, dtype=dtype)
            w = normal(g, D, W, scale=0.6)
            b = normal(g, D, scale=0.5) if full else None
            s = normal(g, N, D, W - 1, dtype=dtype) if full else None
            gf = normal(g, N, D, W - 1, dtype=dtype) if full else None
            flags, lengths = episodes(g, N, T, which)
            kw = dict(state=s, flags=flags, convention=convention_of(which), lengths=lengths,
                      silu=full)
            want = ref.conv(x, w, b, grad_out=go, grad_final=gf, **kw)
            out, final = rl.causal_conv(x, w, b, with_state=True, **kw)
            check(out, want["out"], f"T={T} out")
            check(final, want["final"], f"T={T} final")
            grads = rl.causal_conv_backward(go, x, w, b, grad_state=gf, **kw)
            for name in ("x", "weight", "bias", "state"):
                got = getattr(grads, name)
                if got is not None:
                    check(got, want[name], f"T={T} grad {name}")
            assert (grads.bias is None) == (b is None) and (grads.state is None) == (s is None)


def test_conv_rows_continue(gpu_device):
    """A row in two calls, the state handed on, is the row in one."""
    g = gen(1)
    x, w, b = normal(g, 3, 5, 40), normal(g, 5, 4), normal(g, 5)
    whole, final = rl.causal_conv(x, w, b, with_state=True)
    for cut in (1, 2, 3, 8, 39):
        first, s = rl.causal_conv(x[..., :cut].contiguous(), w, b, with_state=True)
        rest, f = rl.causal_conv(x[..., cut:], w, b, state=s, with_state=True)
        assert torch.equal(torch.cat([first, rest], 2), whole) and torch.equal(f, final)


def test_conv_strided_views(gpu_device):
    g = gen(2)
    for dtype in DTYPES:
        wide = normal(g, 4, 10, 77, dtype=dtype)
        w, b = normal(g, 5, 4), normal(g, 5)
        for x in (wide[:, 3:8, 1:], wide[:, ::2, :70], wide[::2, :5, 5:12],
                  wide[:1, :5].expand(4, 5, 77), wide[:, :1, :33].expand(4, 5, 33)):
            go = torch.zeros(x.shape[0], 9, x.shape[2] + 3, device="cuda", dtype=dtype)
            go = (go + 1)[:, 2:7, 3:]
            out, final = rl.causal_conv(x, w, b, with_state=True)
            out1, final1 = rl.causal_conv(x.contiguous(), w, b, with_state=True)
            assert torch.equal(out, out1) and torch.equal(final, final1)
            a = rl.causal_conv_backward(go, x, w, b)
            c = rl.causal_conv_backward(go.contiguous(), x.contiguous(), w, b)
            for p, q in zip(a, c):
                assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_step(dtype, W, gpu_device):
    # the last: eight channels a thread, workgroups that walk several sequences
    for N, D, slots in ((1, 1, False), (3, 7, False), (5, 64, True), (2, 300, True),
                        (1, 2048, False), (300, 9, True), (520, 4099, True)):
        g = gen(10 + D)
        print(f"conv step {dtype} W={W} {N}x{D} slots={slots}", flush=True)
        places = N + 3
        w, b = normal(g, D, W, scale=0.6), normal(g, D)
        state = normal(g, places, D, W - 1, dtype=dtype)
        before = state.clone()
        x = normal(g, N, D + 5, dtype=dtype)[:, 2:D + 2]
        starts = (torch.rand(N, generator=g, device="cuda") < 0.4).to(torch.uint8)
        at = torch.randperm(places, generator=g, device="cuda")[:N] if slots \
            else torch.arange(N, device="cuda")
        out = rl.causal_conv_step(x, w, b, state, slots=at.int() if slots else None, flags=starts)
        want = ref.conv(x[:, :, None], w, b, before[at], starts[:, None])
        check(out[:, :, None], want["out"], "out")
        check(state[at], want["final"], "state")
        others = torch.ones(places, dtype=torch.bool, device="cuda")
        others[at] = False
        assert torch.equal(state[others], before[others])


# -------------------------------------------------------------------- the scan
def scan_inputs(g, N, ch, S, T, G, dtype, full):
    t = {"u": normal(g, N, ch, T, dtype=dtype), "delta": normal(g, N, ch, T, dtype=dtype),
         "A": -(0.05 + 2 * torch.rand(ch, S, generator=g, device="cuda")),
         "B": normal(g, N, G, S, T, dtype=dtype), "C": normal(g, N, G, S, T, dtype=dtype)}
    if full:
        t.update(D=normal(g, ch), z=normal(g, N, ch, T, dtype=dtype),
                 delta_bias=normal(g, ch) - 2)
    return t


# states on both sides of the eight staged together, channels on both sides of
# the sixteen of a workgroup, steps on both sides of a lane's eight and a tile's 128
SCAN_SHAPES = [(5, 3, 4, 1, 1), (5, 2, 1, 2, 1), (5, 18, 3, 7, 1), (5, 4, 8, 8, 2),
               (2, 17, 9, 9, 1), (5, 6, 16, 33, 3), (2, 34, 17, 64, 2), (5, 3, 16, 127, 1),
               (5, 16, 5, 128, 1), (5, 5, 16, 129, 1), (1, 2, 128, 40, 1), (5, 3, 33, 300, 1),
               (1, 1, 16, 1030, 1)]


def run_scan(t, s, flags, lengths, convention, softplus, go=None, gf=None):
    kw = dict(flags=flags, lengths=lengths, convention=convention, softplus=softplus, state=s)
    y, final, points = rl.selective_scan(**t, with_state=True, with_checkpoints=go is not None,
                                         **kw)
    if go is None:
        return y, final, None
    grads = rl.selective_scan_backward(go, **t, checkpoints=points, grad_state=gf, **kw)
    return y, final, grads


@pytest.mark.parametrize("which", WHICH, ids=lambda w: w.replace(" ", "_") or "plain")
@pytest.mark.parametrize("shape", SCAN_SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_scan(dtype, shape, which, gpu_device):
    N, ch, S, T, G = shape
    for full in (True, False):
        g = gen(1000 + T + S)
        print(f"scan {dtype} {shape} {which!r} full={full}", flush=True)
        t = scan_inputs(g, N, ch, S, T, G, dtype, full)
        if not full:
            t["delta"] = t["delta"].abs() * 0.1  # used as it is
        s = normal(g, N, ch, S) if full else None
        gf = normal(g, N, ch, S) if full else None
        go = normal(g, N, ch, T, dtype=dtype)
        flags, lengths = episodes(g, N, T, which)
        convention = convention_of(which)
        want = ref.scan(**t, state=s, flags=flags, lengths=lengths, convention=convention,
                        softplus=full, grad_y=go, grad_final=gf)
        y, final, grads = run_scan(t, s, flags, lengths, convention, full, go, gf)
        check(y, want["y"], "y")
        check(final, want["final"], "final state")
        for name in grads._fields:
            if getattr(grads, name) is not None:
                check(getattr(grads, name), want[name], f"grad {name}")
        given = [n for n in grads._fields if getattr(grads, n) is not None]
        assert len(given) == (9 if full else 5)


@pytest.mark.parametrize("which", ["", "flags"], ids=lambda w: w or "plain")
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_scan_many_channels(dtype, which, gpu_device):
    """Enough channels that one wave takes four of them alone."""
    N, ch, S, T, G = 4, 3100, 5, 140, 1
    g = gen(31)
    t = scan_inputs(g, N, ch, S, T, G, dtype, True)
    go = normal(g, N, ch, T, dtype=dtype)
    flags, _ = episodes(g, N, T, which)
    want = ref.scan(**t, flags=flags, grad_y=go)
    y, final, grads = run_scan(t, None, flags, None, 0, True, go)
    check(y, want["y"], "y")
    check(final, want["final"], "final state")
    for name in grads._fields:
        if getattr(grads, name) is not None:
            check(getattr(grads, name), want[name], f"grad {name}")


# Rows of few steps, enough of them that four lanes or one take a row, over several
# tiles too; and rows of 16 lanes whose four channels one wave takes alone.
MANY_ROWS = [(20, 1026, 5, 70, 1), (64, 210, 17, 20, 3), (90, 510, 4, 7, 1), (160, 510, 3, 13, 1),
             (4, 3100, 5, 250, 1)]


@pytest.mark.parametrize("which", ["", "flags lengths after"], ids=lambda w: w or "plain")
@pytest.mark.parametrize("shape", MANY_ROWS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_scan_many_rows(dtype, shape, which, gpu_device):
    N, ch, S, T, G = shape
    g = gen(32)
    t = scan_inputs(g, N, ch, S, T, G, dtype, True)
    s, gf, go = normal(g, N, ch, S), normal(g, N, ch, S), normal(g, N, ch, T, dtype=dtype)
    flags, lengths = episodes(g, N, T, which)
    kw = dict(flags=flags, lengths=lengths, convention=convention_of(which))
    want = ref.scan(**t, state=s, grad_y=go, grad_final=gf, **kw)
    y, final, grads = run_scan(t, s, flags, lengths, kw["convention"], True, go, gf)
    check(y, want["y"], "y")
    check(final, want["final"], "final state")
    for name in grads._fields:
        check(getattr(grads, name), want[name], f"grad {name}")


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_scan_extreme_steps(dtype, gpu_device):
    """Step sizes from e^-15 to 15 and decays from 1 (A = 0) to e^-300 a step."""
    g = gen(3)
    N, ch, S, T = 2, 6, 8, 150
    t = scan_inputs(g, N, ch, S, T, 1, dtype, True)
    t["delta"] = normal(g, N, ch, T, dtype=dtype, scale=5.0)
    t["A"] = -torch.tensor([0.0, 1e-6, 1e-3, 0.1, 1.0, 5.0, 20.0, 1e3], device="cuda").expand(
        ch, S).contiguous()
    go = normal(g, N, ch, T, dtype=dtype)
    want = ref.scan(**t, grad_y=go)
    y, final, grads = run_scan(t, None, None, None, 0, True, go)
    check(y, want["y"], "y")
    check(final, want["final"], "final state")
    for name in grads._fields:
        if getattr(grads, name) is not None and name != "state":
            check(getattr(grads, name), want[name], f"grad {name}")


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
@pytest.mark.parametrize("T", [5, 150])
def test_masked_step_sizes(T, dtype, gpu_device):
    """Steps whose delta is the type's lowest value, or -infinity, have size 0:
    they change no state and pass finite gradients; a row may be all such steps."""
    g = gen(41)
    N, ch, S = 4, 18, 6
    t = scan_inputs(g, N, ch, S, T, 1, dtype, True)
    masked = torch.rand(N, 1, T, generator=g, device="cuda") < 0.4
    masked[1], masked[2] = True, False
    masked = masked.expand(N, ch, T)
    t["delta"] = t["delta"].masked_fill(masked, torch.finfo(dtype).min)
    s, gf, go = normal(g, N, ch, S), normal(g, N, ch, S), normal(g, N, ch, T, dtype=dtype)
    want = ref.scan(**t, state=s, grad_y=go, grad_final=gf)
    y, final, grads = run_scan(t, s, None, None, 0, True, go, gf)
    check(y, want["y"], "y")
    check(final, want["final"], "final state")
    assert torch.equal(final[1], s[1])
    for name in grads._fields:
        check(getattr(grads, name), want[name], f"grad {name}")
    inf = dict(t, delta=t["delta"].masked_fill(masked, -float("inf")))
    y2, final2, grads2 = run_scan(inf, s, None, None, 0, True, go, gf)
    assert torch.equal(y2, y) and torch.equal(final2, final)
    assert all(torch.equal(a, b) for a, b in zip(grads2, grads))
    pool = s.clone()
    out = rl.selective_step(t["u"][..., 0].contiguous(), inf["delta"][..., 0].contiguous(),
                            t["A"], t["B"][..., 0].contiguous(), t["C"][..., 0].contiguous(),
                            pool, t["D"], t["z"][..., 0].contiguous(), t["delta_bias"])
    assert torch.equal(pool[1], s[1]) and bool(out.isfinite().all())


def test_scan_rows_continue(gpu_device):
    """A row in two calls, the state handed on, agrees with the row in one."""
    g = gen(4)
    N, ch, S, T = 2, 5, 7, 200
    t = scan_inputs(g, N, ch, S, T, 1, torch.float32, True)
    want = ref.scan(**t)
    for cut in (1, 8, 100, 128, 199):
        def part(a, b):
            return {k: v[..., a:b] if k in ("u", "delta", "z", "B", "C") else v
                    for k, v in t.items()}
        y1, s, _ = rl.selective_scan(**part(0, cut), with_state=True)
        y2, f, _ = rl.selective_scan(**part(cut, T), state=s, with_state=True)
        # each part's rounding, once more for the second's start
        value, bound = want["y"]
        check(torch.cat([y1, y2], 2), (value, 2 * bound), f"cut {cut} y")
        check(f, (want["final"][0], 2 * want["final"][1]), f"cut {cut} state")


def test_scan_strided_views(gpu_device):
    g = gen(5)
    N, ch, S, T, G = 3, 6, 4, 137, 2
    for dtype in DTYPES:
        xz = normal(g, N, 2 * ch + 1, T + 3, dtype=dtype)
        bc = normal(g, N + 1, 2 * G * S, T + 1, dtype=dtype)
        t = {"u": xz[:, :ch, 1:T + 1], "z": xz[:, ch + 1:, 3:],
             "delta": normal(g, ch, N, T, dtype=dtype).transpose(0, 1),
             "A": -torch.rand(ch, S, generator=g, device="cuda"),
             "B": bc[1:, :G * S, 1:].view(N, G, S, T), "C": bc[:N, G * S:, :T].view(N, G, S, T)}
        go = normal(g, N, ch, T + 5, dtype=dtype)[..., 5:]
        a = run_scan(t, None, None, None, 0, True, go)
        c = run_scan({k: v.contiguous() for k, v in t.items()}, None, None, None, 0, True,
                     go.contiguous())
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
        for p, q in zip(a[2], c[2]):
            assert (p is None and q is None) or torch.equal(p, q)
        # one group without its dimension, and one row broadcast to every sequence
        one = dict(t, B=t["B"][:, 0], C=t["C"][:1, 0].expand(N, S, T))
        y, _, _ = rl.selective_scan(**one)
        y1, _, _ = rl.selective_scan(**dict(one, B=one["B"][:, None].contiguous(),
                                            C=one["C"][:, None].contiguous()))
        assert torch.equal(y, y1)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_scan_step(dtype, gpu_device):
    for N, ch, S, G, slots in ((1, 1, 1, 1, False), (3, 6, 4, 2, False), (5, 33, 16, 1, True),
                               (2, 10, 7, 5, True), (1, 2048, 16, 1, False), (40, 8, 128, 2, True),
                               (3, 5, 65, 1, True), (70, 4100, 16, 2, True)):
        g = gen(20 + S)
        print(f"scan step {dtype} {N}x{ch}x{S} G={G} slots={slots}", flush=True)
        places = N + 2
        t = scan_inputs(g, N, ch, S, 1, G, dtype, True)
        state = normal(g, places, ch, S)
        before = state.clone()
        starts = (torch.rand(N, generator=g, device="cuda") < 0.4).to(torch.uint8)
        at = torch.randperm(places, generator=g, device="cuda")[:N] if slots \
            else torch.arange(N, device="cuda")
        step = {k: v[..., 0] if k in ("u", "delta", "z", "B", "C") else v for k, v in t.items()}
        # rows of a wider projection
        step["u"] = torch.cat([step["u"], step["z"]], 1)[:, :ch]
        y = rl.selective_step(state=state, slots=at.int() if slots else None, flags=starts, **{
            k: v if k == "u" else v.contiguous() for k, v in step.items()})
        want = ref.scan(**t, state=before[at], flags=starts[:, None])
        check(y[:, :, None], want["y"], "y")
        check(state[at], want["final"], "state")
        others = torch.ones(places, dtype=torch.bool, device="cuda")
        others[at] = False
        assert torch.equal(state[others], before[others])


def test_empty_seats(gpu_device):
    """Slots out of range touch nothing and give 0."""
    g = gen(6)
    for dtype in DTYPES:
        slots = torch.tensor([2, -1, 7, 0, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                             device="cuda")
        real = torch.tensor([0, 3], device="cuda")
        N, D = 6, 70
        state = normal(g, 7, D, 3, dtype=dtype)
        before = state.clone()
        out = rl.causal_conv_step(normal(g, N, D, dtype=dtype), normal(g, D, 4), None, state,
                                  slots=slots)
        empty = [1, 2, 4, 5]
        assert not out[empty].any() and out[real].any()
        untouched = [1, 3, 4, 5, 6]
        assert torch.equal(state[untouched], before[untouched])
        t = scan_inputs(g, N, D, 5, 1, 1, dtype, True)
        t = {k: v[..., 0].contiguous() if k in ("u", "delta", "z", "B", "C") else v
             for k, v in t.items()}
        pool = normal(g, 7, D, 5)
        before = pool.clone()
        y = rl.selective_step(state=pool, slots=slots, **t)
        assert not y[empty].any() and y[real].any()
        assert torch.equal(pool[untouched], before[untouched])


def test_steps_follow_rows(gpu_device):
    """Rows for a prompt, then single steps, agree with the whole as rows."""
    g = gen(7)
    N, ch, S, W, P, T = 3, 40, 16, 4, 19, 27
    t = scan_inputs(g, N, ch, S, T, 1, torch.float32, True)
    x, w, b = t["u"], normal(g, ch, W, scale=0.5), normal(g, ch)
    out, _ = rl.causal_conv(x, w, b)
    whole = ref.scan(**dict(t, u=out))
    _, cs = rl.causal_conv(x[..., :P], w, b, with_state=True)
    rows = {k: v[..., :P] if k in ("delta", "z", "B", "C") else v for k, v in t.items()}
    _, hs, _ = rl.selective_scan(**dict(rows, u=out[..., :P]), with_state=True)
    value, bound = whole["y"]
    for i in range(P, T):
        c = rl.causal_conv_step(x[:, :, i].contiguous(), w, b, cs)
        assert torch.allclose(c, out[:, :, i], rtol=2e-6, atol=1e-6)
        step = {k: v[..., i].contiguous() if k in ("delta", "z", "B", "C") else v
                for k, v in t.items()}
        y = rl.selective_step(state=hs, **dict(step, u=out[:, :, i].contiguous()))
        check(y, (value[:, :, i], 3 * bound[:, :, i]), f"step {i}")


# ------------------------------------------------------------ what may not pass
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nothing_passes_an_episode_start(bad, gpu_device):
    """Steps 20..29 of a row are poisoned in every input; the episodes before
    and after, other rows and other sequences stay bit for bit."""
    g = gen(8)
    N, ch, S, T = 3, 18, 6, 150
    for dtype in (torch.float32, torch.bfloat16):
        t = scan_inputs(g, N, ch, S, T, 1, dtype, True)
        x, w, go = normal(g, N, ch, T, dtype=dtype), normal(g, ch, 4), normal(g, N, ch, T,
                                                                              dtype=dtype)
        flags = torch.zeros(N, T, dtype=torch.uint8, device="cuda")
        flags[1, 20] = flags[1, 30] = 1

        def run(t, x, go):
            y, final, points = rl.selective_scan(**t, flags=flags, with_state=True,
                                                 with_checkpoints=True)
            gr = rl.selective_scan_backward(go, **t, checkpoints=points, flags=flags)
            o, f = rl.causal_conv(x, w, flags=flags, with_state=True)
            cg = rl.causal_conv_backward(go, x, w, flags=flags)
            return {"y": y, "gu": gr.u, "gdelta": gr.delta, "gz": gr.z, "out": o, "gx": cg.x,
                    "gB": gr.B, "gC": gr.C}, {"final": final, "fc": f}

        rows, ends = run(t, x, go)
        t2 = {k: v.clone() for k, v in t.items()}
        for k in ("u", "delta", "z", "B", "C"):
            t2[k][1, ..., 20:30] = bad
        x2, go2 = x.clone(), go.clone()
        x2[1, :, 20:30] = bad
        go2[1, :, 20:30] = bad
        rows2, ends2 = run(t2, x2, go2)
        for k, v in rows.items():
            a, b = v.clone(), rows2[k].clone()
            a[1, ..., 20:30] = 0
            b[1, ..., 20:30] = 0
            assert torch.equal(a, b), k
        for k, v in ends.items():
            assert torch.equal(v, ends2[k]), k


@pytest.mark.parametrize("shape", [(200, 510, 3, 13), (40, 1026, 5, 70)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nothing_passes_an_episode_start_in_many_rows(bad, shape, gpu_device):
    """Where one lane or four take a row: steps 5..9 are poisoned."""
    N, ch, S, T = shape
    g = gen(18)
    t = scan_inputs(g, N, ch, S, T, 1, torch.float32, True)
    go = normal(g, N, ch, T)
    flags = torch.zeros(N, T, dtype=torch.uint8, device="cuda")
    flags[1, 5] = flags[1, 10] = 1

    def run(t, go):
        y, final, points = rl.selective_scan(**t, flags=flags, with_state=True,
                                             with_checkpoints=True)
        gr = rl.selective_scan_backward(go, **t, checkpoints=points, flags=flags)
        return {"y": y, "gu": gr.u, "gdelta": gr.delta, "gz": gr.z, "gB": gr.B, "gC": gr.C}, final

    rows, final = run(t, go)
    t2, go2 = {k: v.clone() for k, v in t.items()}, go.clone()
    for v in (t2["u"], t2["delta"], t2["z"], t2["B"], t2["C"], go2):
        v[1, ..., 5:10] = bad
    rows2, final2 = run(t2, go2)
    for k, v in rows.items():
        v[1, ..., 5:10] = rows2[k][1, ..., 5:10] = 0
        assert torch.equal(v, rows2[k]), k
    assert torch.equal(final, final2)


def test_nothing_enters_past_a_rows_length(gpu_device):
    g = gen(9)
    N, ch, S, T = 4, 18, 6, 150
    lengths = torch.tensor([0, 1, 130, 150], dtype=torch.int32, device="cuda")
    past = torch.arange(T, device="cuda") >= lengths[:, None]
    t = scan_inputs(g, N, ch, S, T, 1, torch.float32, True)
    x, w, go = normal(g, N, ch, T), normal(g, ch, 4), normal(g, N, ch, T)
    s, cs = normal(g, N, ch, S), normal(g, N, ch, 3)

    def run(t, x, go):
        y, final, points = rl.selective_scan(**t, state=s, lengths=lengths, with_state=True,
                                             with_checkpoints=True)
        gr = rl.selective_scan_backward(go, **t, checkpoints=points, state=s, lengths=lengths)
        o, f = rl.causal_conv(x, w, state=cs, lengths=lengths, with_state=True)
        cg = rl.causal_conv_backward(go, x, w, state=cs, lengths=lengths)
        return [y, final, o, f] + [v for v in list(gr) + list(cg) if v is not None]

    clean = run(t, x, go)
    t2 = {k: v.clone() for k, v in t.items()}
    x2, go2 = x.clone(), go.clone()
    for v in (t2["u"], t2["delta"], t2["z"], t2["B"][:, 0], t2["C"][:, 0], x2, go2):
        v.masked_fill_(past[:, None].expand(v.shape), float("nan"))
    for a, b in zip(clean, run(t2, x2, go2)):
        assert torch.equal(a, b)
    for v in (clean[0], clean[2]):
        assert not v.masked_select(past[:, None].expand(v.shape)).any()


# -------------------------------------------------------------- the caller's side
def test_repeats_streams_and_graphs(gpu_device):
    """Bit for bit the same on every call, on another stream, and on every
    replay of a captured graph (with eager work between)."""
    g = gen(11)
    N, ch, S, T = 3, 40, 16, 300
    t = scan_inputs(g, N, ch, S, T, 2, torch.bfloat16, True)
    go = normal(g, N, ch, T, dtype=torch.bfloat16)
    w, b = normal(g, ch, 4), normal(g, ch)
    flags = (torch.rand(N, T, generator=g, device="cuda") < 0.02).to(torch.uint8)
    tensors = [normal(g, n) for n in (1, 700, 5000, 33)]
    outs = [torch.empty_like(v) for v in tensors]
    state0, pool0 = normal(g, N, ch, 3, dtype=torch.bfloat16), normal(g, N, ch, S)
    state, pool = state0.clone(), pool0.clone()
    step = {k: v[..., 0].contiguous() if k in ("u", "delta", "z", "B", "C") else v
            for k, v in t.items()}

    def work():
        state.copy_(state0)
        pool.copy_(pool0)
        c, cf = rl.causal_conv(t["u"], w, b, flags=flags, with_state=True)
        y, f, p = rl.selective_scan(**t, flags=flags, with_state=True, with_checkpoints=True)
        gs = rl.selective_scan_backward(go, **t, checkpoints=p, flags=flags)
        gc = rl.causal_conv_backward(go, t["u"], w, b, flags=flags)
        n = rl.clip_grad_norm(tensors, 0.5, out=outs)
        s1 = rl.causal_conv_step(step["u"], w, b, state)
        s2 = rl.selective_step(state=pool, **step)
        return [v for v in [c, cf, y, f, n, s1, s2, state, pool] + list(gs) + list(gc) + outs
                if v is not None]

    first = [v.clone() for v in work()]
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first, work()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = work()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for rep in range(4):
        for v in captured:
            v.fill_(7.0)
        torch.cumsum(torch.randn(1 << 16, device="cuda"), 0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, captured)), f"replay {rep}"


def test_empty_calls(gpu_device):
    w, A = torch.ones(4, 3, device="cuda"), -torch.ones(4, 2, device="cuda")
    for N, T in ((0, 5), (2, 0), (0, 0)):
        x = torch.zeros(N, 4, T, device="cuda")
        s = torch.ones(N, 4, 2, device="cuda")
        out, f = rl.causal_conv(x, w, state=s, with_state=True)
        assert out.shape == x.shape and torch.equal(f, s)
        gr = rl.causal_conv_backward(x, x, w, state=s, grad_state=2 * s)
        assert not gr.weight.any() and torch.equal(gr.state, 2 * s)
        B = torch.zeros(N, 2, T, device="cuda")
        y, f, p = rl.selective_scan(x, x, A, B, B, state=s, with_state=True,
                                    with_checkpoints=True)
        assert y.shape == x.shape and torch.equal(f, s)
        gr = rl.selective_scan_backward(x, x, x, A, B, B, p, state=s, grad_state=2 * s)
        assert not gr.A.any() and torch.equal(gr.state, 2 * s)


def test_offsets_past_32_bits(gpu_device):
    """A sequence that begins past 2^31 elements, and rows whose last channel does."""
    T, ch, S = 1000, 2, 2
    far = (1 << 31) + 1024
    buf = torch.zeros(far + 4 * ch * T, dtype=torch.bfloat16, device="cuda")
    g = gen(12)
    x = buf.as_strided((2, ch, T), (far, T, 1))
    x.copy_(normal(g, 2, ch, T))
    assert x.storage_offset() == 0 and x.stride(0) == far
    w = normal(g, ch, 3)
    assert torch.equal(rl.causal_conv(x, w)[0], rl.causal_conv(x.contiguous(), w)[0])
    rows = buf.as_strided((1, 2, T), (0, far, 1))
    A = -torch.rand(ch, S, generator=g, device="cuda")
    a = rl.selective_scan(rows, rows, A, x[:1, :, :], x[1:, :, :])[0]
    c = rl.selective_scan(rows.contiguous(), rows.contiguous(), A, x[:1].contiguous(),
                          x[1:].contiguous())[0]
    assert torch.equal(a, c)
    p = rl.causal_conv_backward(x, x, w)
    q = rl.causal_conv_backward(x.contiguous(), x.contiguous(), w)
    assert torch.equal(p.x, q.x) and torch.equal(p.weight, q.weight)


def test_refusals(gpu_device):
    x, w = torch.zeros(2, 4, 9, device="cuda"), torch.zeros(4, 3, device="cuda")
    A, B = torch.zeros(4, 2, device="cuda"), torch.zeros(2, 2, 9, device="cuda")
    ok = dict(u=x, delta=x, A=A, B=B, C=B)
    bad_conv = [
        (ValueError, dict(x=x.cpu())), (ValueError, dict(x=x[0])), (TypeError, dict(x=x.int())),
        (ValueError, dict(x=x.transpose(1, 2))), (ValueError, dict(weight=w[:3])),
        (ValueError, dict(weight=w[:, :1].contiguous())), (TypeError, dict(weight=w.half())),
        (ValueError, dict(weight=None)), (ValueError, dict(bias=w[0])),
        (ValueError, dict(state=x)), (TypeError, dict(flags=x[:, 0].contiguous())),
        (ValueError, dict(flags=torch.zeros(2, 8, dtype=torch.uint8, device="cuda"))),
        (TypeError, dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))),
        (ValueError, dict(out=x[:1])), (rl.RlcaError, dict(out=x)),
        (rl.RlcaError, dict(convention=5)),
    ]
    for error, change in bad_conv:
        with pytest.raises(error):
            rl.causal_conv(**{**dict(x=x, weight=w), **change})
    bad_scan = [
        (ValueError, dict(delta=x[..., :8])), (TypeError, dict(delta=x.half())),
        (ValueError, dict(A=A[0])), (ValueError, dict(A=torch.zeros(4, 129, device="cuda"))),
        (TypeError, dict(A=A.double())), (ValueError, dict(B=None)), (ValueError, dict(B=B[0])),
        (ValueError, dict(B=torch.zeros(2, 3, 2, 9, device="cuda"),
                          C=torch.zeros(2, 3, 2, 9, device="cuda"))),
        (ValueError, dict(C=torch.zeros(2, 2, 2, 9, device="cuda"))),
        (ValueError, dict(z=x[:1])), (ValueError, dict(D=A)), (ValueError, dict(delta_bias=A)),
        (TypeError, dict(state=torch.zeros(2, 4, 2, device="cuda").half())),
        (rl.RlcaError, dict(y=x)), (rl.RlcaError, dict(convention=-1)),
    ]
    for error, change in bad_scan:
        with pytest.raises(error):
            rl.selective_scan(**{**ok, **change})
    with pytest.raises(ValueError):
        rl.selective_scan_backward(x, **ok, checkpoints=A)
    with pytest.raises(ValueError):
        rl.selective_scan_backward(x, **ok, checkpoints=None)
    xs, state = x[:, :, 0].contiguous(), torch.zeros(1, 4, 2, device="cuda")
    with pytest.raises(ValueError):
        rl.causal_conv_step(xs, w, None, state)          # one place, two sequences
    with pytest.raises(TypeError):
        rl.causal_conv_step(xs, w, None, state, slots=torch.zeros(2, dtype=torch.int64,
                                                                  device="cuda"))
    with pytest.raises(ValueError):
        rl.selective_step(xs, xs, A, B[..., 0].contiguous(), B[..., 0].contiguous(), state)
