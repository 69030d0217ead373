"""How the block and beam operators are called: what the binding refuses, outputs that
the caller brings, several threads and streams, graphs replayed in turn, the same
results from the same inputs, inputs far apart in memory, and what may not pass an
episode's start in rows that waves share."""
import threading

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_gated_gpu import inputs
from .test_sequence_gpu import gen, normal

pytestmark = pytest.mark.gpu


def calls(g, dtype=torch.bfloat16):
    """Closures that run every operator, each with inputs of its own."""
    a = inputs(g, 2, 130, 2100, dtype, True)
    go = normal(g, 2, 130, 2100, dtype=dtype)
    args = (a["x"], a["input_gate"], a["decay_gate"], a["decay"])
    kw = dict(input_bias=a["input_bias"], decay_bias=a["decay_bias"], state=a["state"])

    def gated():
        out, f, c = rl.gated_recurrence(*args, with_state=True, with_checkpoints=True, **kw)
        return out, f, *rl.gated_recurrence_backward(go, *args, c, **kw)

    x, w = normal(g, 2, 700, 300, dtype=dtype), normal(g, 700)

    def norm():
        out, s = rl.rms_norm(x, w, x)
        q, scale, _ = rl.rms_norm_8bit(x, w)
        return out, s, q.float(), scale, *rl.rms_norm_backward(out, s, w, grad_sum=x)

    logits, scores = normal(g, 3, 4, 9001, dtype=dtype), normal(g, 3, 4)
    slots = torch.arange(12, device="cuda", dtype=torch.int32).view(3, 4)
    pool = normal(g, 12, 5000)

    def beams():
        choice = rl.beam_select(logits, scores)
        mine = [pool.clone()]
        return *choice, rl.beam_reorder(mine, slots, choice.parents), *mine

    return [gated, norm, beams]


def test_results_are_reproducible(gpu_device):
    for run in calls(gen(1)):
        want = run()
        for _ in range(3):
            for p, q in zip(run(), want):
                assert torch.equal(p, q)


def test_threads_and_streams(gpu_device):
    runs = calls(gen(2))
    want = [run() for run in runs]
    torch.cuda.synchronize()
    bad = []

    def work(i, stream):
        with torch.cuda.stream(stream):
            for k in range(12):
                j = (i + k) % len(runs)
                got = runs[j]()
                stream.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want[j])):
                    bad.append((i, j))

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(i, shared if i < 2 else torch.cuda.Stream()))
               for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_graphs_replayed_in_turn(gpu_device):
    """Two graphs of the same calls, captured apart, replayed on two streams at once."""
    runs = calls(gen(3))
    want = [run() for run in runs]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                got = [run() for run in runs]
            graphs.append((graph, got))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        runs[0]()
        torch.cuda.synchronize()
        for _, got in graphs:
            for p, q in zip(got, want):
                assert all(torch.equal(a, b) for a, b in zip(p, q))
                for t in p:
                    t.zero_()
        torch.cuda.synchronize()


def test_outputs_of_the_caller(gpu_device):
    g = gen(4)
    a = inputs(g, 2, 5, 30, torch.float32, False)
    args = (a["x"], a["input_gate"], a["decay_gate"], a["decay"])
    out, final = torch.empty_like(a["x"]), torch.empty(2, 5, device="cuda")
    before = out._version, final._version
    got = rl.gated_recurrence(*args, out=out, final_state=final)
    assert got[0] is out and got[1] is final
    assert out._version > before[0] and final._version > before[1]
    want = rl.gated_recurrence(*args, with_state=True)
    assert torch.equal(out, want[0]) and torch.equal(final, want[1])
    x = a["x"]
    y, s = torch.empty_like(x), torch.empty_like(x)
    got = rl.rms_norm(x, residual=x, out=y, total=s)
    assert got[0] is y and got[1] is s and y._version > 0 and s._version > 0
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(2, 30, device="cuda")
    got = rl.rms_norm_8bit(x, out=q, scale=scale)
    assert got[0] is q and got[1] is scale and scale._version > 0
    state = torch.zeros(2, 5, device="cuda")
    out = torch.empty(2, 5, device="cuda")
    step = [t[:, :, 0].contiguous() for t in args[:3]]
    assert rl.gated_step(*step, a["decay"], state, out=out) is out
    assert out._version > 0 and state._version > 0
    slots = torch.arange(4, device="cuda", dtype=torch.int32).view(2, 2)
    new = torch.empty_like(slots)
    assert rl.beam_reorder([state[:0]], slots, slots % 2, out=new) is new and new._version > 0


def test_what_the_binding_refuses(gpu_device):
    x = torch.zeros(2, 5, 30, device="cuda")
    d = torch.zeros(5, device="cuda")
    step = torch.zeros(2, 5, device="cuda")
    state = torch.zeros(2, 5, device="cuda")
    half, cpu, bad = x.half(), x.cpu(), x[:, :4]
    gated = [dict(x=x.double()), dict(x=x.transpose(1, 2)), dict(input_gate=half),
             dict(decay_gate=cpu), dict(decay_gate=bad), dict(decay=d.half()), dict(decay=d[:4]),
             dict(decay=None), dict(input_bias=d[:3]), dict(state=state.half()),
             dict(flags=torch.zeros(2, 29, device="cuda", dtype=torch.uint8)),
             dict(flags=torch.zeros(2, 30, device="cuda")),
             dict(lengths=torch.zeros(2, device="cuda", dtype=torch.int64)),
             dict(out=half), dict(out=x.transpose(1, 2).contiguous().transpose(1, 2)),
             dict(final_state=state[:1])]
    for change in gated:
        with pytest.raises((TypeError, ValueError)):
            rl.gated_recurrence(**{**dict(x=x, input_gate=x, decay_gate=x, decay=d), **change})
    for scale in (0.0, -8.0, float("nan"), float("inf")):
        with pytest.raises(rl.RlcaError, match="VALUE"):
            rl.gated_recurrence(x, x, x, d, scale=scale)
        with pytest.raises(rl.RlcaError, match="VALUE"):
            rl.gated_step(step, step, step, d, state, scale=scale)
    with pytest.raises(rl.RlcaError, match="ALIAS"):
        rl.gated_recurrence(x, x, x, d, out=x)
    with pytest.raises(rl.RlcaError, match="VALUE"):
        rl.gated_recurrence(x, x, x, d, convention=5)
    points = rl.gated_recurrence(x, x, x, d, with_checkpoints=True)[2]
    for change in (dict(grad_out=half), dict(checkpoints=None), dict(checkpoints=points[:-1]),
                   dict(grad_state=state[:1])):
        with pytest.raises((TypeError, ValueError)):
            rl.gated_recurrence_backward(**{**dict(grad_out=x, x=x, input_gate=x, decay_gate=x,
                                                   decay=d, checkpoints=points), **change})
    for change in (dict(state=None), dict(state=state[:1]), dict(state=state.half()),
                   dict(slots=torch.zeros(2, device="cuda")), dict(input_gate=step[:1])):
        with pytest.raises((TypeError, ValueError)):
            rl.gated_step(**{**dict(x=step, input_gate=step, decay_gate=step, decay=d,
                                    state=state), **change})
    for f in (rl.rms_norm, rl.rms_norm_8bit):
        for change in (dict(x=x.double()), dict(weight=d.half()), dict(weight=d[:2]),
                       dict(residual=half), dict(residual=bad), dict(total=x),
                       dict(out=x.double()), dict(lengths=torch.zeros(2, device="cuda"))):
            with pytest.raises((TypeError, ValueError)):
                f(**{**dict(x=x), **change})
        for eps in (0.0, -1.0, float("nan")):
            with pytest.raises(rl.RlcaError, match="VALUE"):
                f(x, eps=eps)
    with pytest.raises(rl.RlcaError, match="ALIAS"):
        rl.rms_norm(x, residual=half.float(), total=x)
    for change in (dict(grad_out=None), dict(grad_out=half), dict(grad_sum=bad)):
        with pytest.raises((TypeError, ValueError)):
            rl.rms_norm_backward(**{**dict(grad_out=x, x=x), **change})
    scores = torch.zeros(2, 5, device="cuda")
    for change in (dict(logits=x.double()), dict(logits=x.transpose(1, 2)), dict(scores=None),
                   dict(scores=scores.half()), dict(scores=scores[:1]), dict(picks=0),
                   dict(picks=65), dict(picks=151, logits=x), dict(finished=scores),
                   dict(logits=torch.zeros(2, 65, 3, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            rl.beam_select(**{**dict(logits=x, scores=scores), **change})
    for pad in (-1, 30):
        with pytest.raises(rl.RlcaError, match="VALUE"):
            rl.beam_select(x, scores, finished=scores.bool(), pad_token=pad)
    slots = torch.arange(4, device="cuda", dtype=torch.int32).view(2, 2)
    for pools, change in (([state, state[:1]], {}), ([x.transpose(0, 2)], {}), ([cpu], {}),
                          ([state], dict(parents=slots.long())), ([state], dict(parents=None)),
                          ([state], dict(parents=slots[:1])), ([state], dict(slots=slots.long())),
                          ([state], dict(out=slots[:1]))):
        with pytest.raises((TypeError, ValueError)):
            rl.beam_reorder(**{**dict(pools=pools, slots=slots, parents=slots % 2), **change})
    with pytest.raises(rl.RlcaError, match="ALIAS"):
        rl.beam_reorder([state, state], slots, slots % 2)


def test_nothing_passes_a_start_in_shared_rows(gpu_device):
    """As for rows that waves walk alone: NaN and infinity before an episode's start, in
    rows that the waves of a workgroup share and in whole-wave rows of several tiles."""
    for N, D, T in ((1, 110, 4300), (3, 40, 1400)):
        for dtype in (torch.float32, torch.bfloat16):
            g = gen(T)
            a = inputs(g, N, D, T, dtype, True)
            go, gf = normal(g, N, D, T, dtype=dtype), normal(g, N, D)
            for cut in (1, 512, 1027, T - 2):
                flags = torch.zeros(N, T, device="cuda", dtype=torch.uint8)
                flags[:, cut] = 1

                def run(x, go, state):
                    args = (x, a["input_gate"], a["decay_gate"], a["decay"])
                    out, final, c = rl.gated_recurrence(*args, state=state, flags=flags,
                                                        with_state=True, with_checkpoints=True)
                    return out, final, rl.gated_recurrence_backward(
                        go, *args, c, state=state, flags=flags, grad_state=gf)

                want = run(a["x"], go, a["state"])
                for bad in (float("nan"), float("inf")):
                    x, s, late = a["x"].clone(), a["state"].clone(), go.clone()
                    x[:, :, :cut] = bad
                    s[:] = bad
                    got = run(x, go, s)
                    assert torch.equal(got[0][:, :, cut:], want[0][:, :, cut:])
                    assert torch.equal(got[1], want[1])
                    for name in ("x", "input_gate", "decay_gate"):
                        assert torch.equal(getattr(got[2], name)[:, :, cut:],
                                           getattr(want[2], name)[:, :, cut:])
                    late[:, :, cut:] = bad
                    got = run(a["x"], late, a["state"])
                    assert torch.equal(got[2].state, want[2].state)
                    for name in ("x", "input_gate", "decay_gate"):
                        assert torch.equal(getattr(got[2], name)[:, :, :cut],
                                           getattr(want[2], name)[:, :, :cut])


def test_inputs_far_apart(gpu_device):
    """Sequences more than 2^32 elements apart."""
    far = (1 << 32) + 8
    wide = torch.zeros(far + 4000, dtype=torch.float16, device="cuda")
    g = gen(6)

    def place(t):
        n, *shape = t.shape
        at = wide[:far + t[0].numel()].as_strided(t.shape, (far, *t[0].stride()))
        at.copy_(t)
        return at

    x = normal(g, 2, 4, 200, dtype=torch.float16)
    decay = torch.linspace(-6, 0, 4, device="cuda")
    out, _, c = rl.gated_recurrence(place(x), x, x, decay, with_checkpoints=True)
    want = rl.gated_recurrence(x, x, x, decay)[0]
    assert torch.equal(out, want)
    grads = rl.gated_recurrence_backward(place(x), x, x, x, decay, c)
    plain = rl.gated_recurrence_backward(x, x, x, x, decay, c)
    assert all(torch.equal(p, q) for p, q in zip(grads, plain) if p is not None)
    w = normal(g, 4)
    assert torch.equal(rl.rms_norm(place(x), w)[0], rl.rms_norm(x, w)[0])
    assert torch.equal(rl.rms_norm_backward(place(x), x, w).x, rl.rms_norm_backward(x, x, w).x)
    row = normal(g, 2, 3000, dtype=torch.float16)
    assert torch.equal(rl.rms_norm(place(row))[0], rl.rms_norm(row)[0])
    steps = [rl.gated_step(r, row, row, w[:1].expand(3000).contiguous(),
                           torch.zeros(2, 3000, device="cuda")) for r in (place(row), row)]
    assert torch.equal(*steps)
    logits = normal(g, 2, 3, 1300, dtype=torch.float16)
    scores = torch.zeros(2, 3, device="cuda")
    for p, q in zip(rl.beam_select(place(logits), scores), rl.beam_select(logits, scores)):
        assert torch.equal(p, q)
