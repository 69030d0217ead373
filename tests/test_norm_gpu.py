"""The root-mean-square norm's kernels against the 64-bit reference, each output
within the bound that the reference carries for float32 arithmetic plus one rounding
to its type (blocks_reference.py): storage types, channels on both sides of what a
thread keeps, rows of one step, of odd and of many, dense rows of channels, lengths
from 0, strides, values whose squares overflow, and what lies past a row's end."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import blocks_reference as ref
from .test_sequence_gpu import DTYPES, NAMES, check, episodes, gen, normal

pytestmark = pytest.mark.gpu

# threads of 4, 8 and 16 channels, channels that are read twice, few and many tiles,
# one step a row (dense rows of channels: a wave or a workgroup each, or more)
SHAPES = [(5, 1, 1), (5, 3, 2), (5, 70, 7), (5, 128, 65), (2, 129, 33), (3, 200, 130),
          (2, 1100, 40), (1, 2051, 9), (260, 300, 33), (130, 1030, 70), (1, 8200, 17),
          (9, 64, 1), (7, 2048, 1), (5, 2049, 1), (3, 8195, 1), (1030, 65, 1), (2, 20000, 1),
          (70, 129, 520)]


def check_all(x, w, res, go, gs, lengths):
    dims = x.dim()
    want = ref.rms_norm(x, w, res, lengths=lengths, grad_out=go, grad_sum=gs)
    out, total = rl.rms_norm(x, w, res, lengths=lengths)
    check(out, want["out"], "out")
    s = x
    if res is not None:
        assert torch.equal(total.cpu().double(), want["sum"][0])
        s = total
    else:
        assert total is None
    q, scale, total8 = rl.rms_norm_8bit(x, w, res, lengths=lengths)
    assert q.dtype == torch.float8_e4m3fn
    check(scale, want["scale"], "scale")
    check(q.cpu().double() * scale.cpu().double().unsqueeze(1), want["dequantized"], "8 bits")
    assert res is None or torch.equal(total8, total)
    grads = rl.rms_norm_backward(go, s, w, grad_sum=gs, lengths=lengths)
    check(grads.x, want["x"], "grad x")
    if w is None:
        assert grads.weight is None
    else:
        check(grads.weight, want["weight"], "grad weight")
    assert dims == out.dim() == grads.x.dim()


@pytest.mark.parametrize("which", ["", "lengths"], ids=["plain", "lengths"])
@pytest.mark.parametrize("full", [True, False], ids=["full", "bare"])
@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_norm(dtype, full, which, gpu_device):
    for N, D, T in SHAPES:
        g = gen(100 + T + D)
        print(f"norm {dtype} {which!r} {N}x{D}x{T} full={full}", flush=True)
        x, go = normal(g, N, D, T, dtype=dtype), normal(g, N, D, T, dtype=dtype)
        w = 1 + normal(g, D, scale=0.3) if full else None
        res = normal(g, N, D, T, dtype=dtype, scale=2.0) if full else None
        gs = normal(g, N, D, T, dtype=dtype) if full else None
        check_all(x, w, res, go, gs, episodes(g, N, T, which)[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_norm_of_single_steps(dtype, gpu_device):
    """[num_seqs, channels], as views of a wider array too, and with rows left out."""
    for N, D in ((1, 4096), (4, 7), (300, 640), (3, 5001)):
        g = gen(D)
        wide = normal(g, N, 4 * D + 3, dtype=dtype)
        x, res, go, gs = (wide[:, i * D + min(i, 3):(i + 1) * D + min(i, 3)] for i in range(4))
        w = normal(g, D)
        check_all(x, w, res, go, gs, None)
        lengths = (torch.arange(N, device="cuda") % 3 - 1).to(torch.int32)
        check_all(x, w, res, go, gs, lengths)


def test_norm_strided_views(gpu_device):
    g = gen(2)
    for dtype in DTYPES:
        for T in (70, 1):
            wide = normal(g, 4, 40, T + 9, dtype=dtype)
            w = normal(g, 10)
            for x, res in ((wide[:, :10, 1:T + 1], wide[:, 10:40:3, 3:T + 3]),
                           (wide[:1, :10, :T].expand(4, 10, T), wide[:, :1, :T].expand(4, 10, T))):
                for a, b in zip(rl.rms_norm(x, w, res), rl.rms_norm(x.contiguous(), w,
                                                                    res.contiguous())):
                    if T > 1:  # the same kernel
                        assert torch.equal(a, b)
                    else:
                        torch.testing.assert_close(a, b)
                go = wide[:, 5:15, 2:T + 2]
                a = rl.rms_norm_backward(go, x, w, grad_sum=res)
                b = rl.rms_norm_backward(go.contiguous(), x.contiguous(), w,
                                         grad_sum=res.contiguous())
                if T > 1:
                    assert torch.equal(a.x, b.x) and torch.equal(a.weight, b.weight)
                else:
                    torch.testing.assert_close(a.x, b.x)
                    torch.testing.assert_close(a.weight, b.weight)


@pytest.mark.parametrize("T", [1, 40])
def test_norm_of_large_values(T, gpu_device):
    """Squares past float32's range, in one step of a tile and in all."""
    for dtype in (torch.float32, torch.bfloat16):
        for D in (70, 300, 2500):
            for steps in (slice(0, 1), slice(None)):
                g = gen(D)
                x = normal(g, 3, D, T, dtype=dtype)
                # below 2^125, so that r is a normal number
                x[1, :, steps] *= 2.0 ** 118
                w, go = normal(g, D), normal(g, 3, D, T, dtype=dtype)
                check_all(x, w, None, go, None, None)


def test_norm_of_zeros(gpu_device):
    for shape in ((2, 40, 9), (2, 40)):
        x = torch.zeros(shape, device="cuda")
        q, scale, _ = rl.rms_norm_8bit(x)
        assert not q.float().any() and bool((scale == 2.0 ** -120).all())
        out, _ = rl.rms_norm(x, residual=x)
        assert not out.any()
        g = rl.rms_norm_backward(torch.ones_like(x), x, eps=1e-4)
        # half of eps's rounding, and the root's reciprocal: four roundings
        torch.testing.assert_close(g.x, torch.full_like(x, 100.0), rtol=4 * 2.0 ** -24, atol=0)


def test_norm_empty(gpu_device):
    for shape in ((0, 3, 9), (3, 0, 9), (3, 5, 0), (0, 5), (3, 0)):
        x = torch.zeros(shape, device="cuda")
        w = torch.ones(shape[1], device="cuda")
        out, total = rl.rms_norm(x, w, x)
        assert out.shape == total.shape == shape
        grads = rl.rms_norm_backward(x, x, w)
        assert grads.x.shape == shape and not grads.weight.any()
        q, scale, _ = rl.rms_norm_8bit(x, w)
        assert q.shape == shape and scale.shape == shape[:1] + shape[2:]


@pytest.mark.parametrize("T", [1, 9, 70])
def test_norm_of_infinities_and_nans(T, gpu_device):
    """In one step: that step's output as the formula says, the others' untouched; past
    a row's length: nothing."""
    for dtype in DTYPES:
        for D in (20, 300):
            g = gen(D)
            x, go = normal(g, 4, D, T, dtype=dtype), normal(g, 4, D, T, dtype=dtype)
            w = normal(g, D)
            lengths = torch.tensor([T, T - 1, T, T], device="cuda", dtype=torch.int32)
            want = (rl.rms_norm(x, w, lengths=lengths)[0],
                    *rl.rms_norm_8bit(x, w, lengths=lengths)[:2],
                    *rl.rms_norm_backward(go, x, w, lengths=lengths))
            for bad in (float("nan"), float("inf")):
                y, go1 = x.clone(), go.clone()
                y[1, D // 2, T - 1] = bad
                go1[1, :, T - 1] = bad
                got = (rl.rms_norm(y, w, lengths=lengths)[0],
                       *rl.rms_norm_8bit(y, w, lengths=lengths)[:2],
                       *rl.rms_norm_backward(go1, y, w, lengths=lengths))
                for p, q in zip(got, want):
                    assert torch.equal(p.float(), q.float())
                y = x.clone()
                y[2, D // 2, T // 2] = bad
                out = rl.rms_norm(y, w, lengths=lengths)[0]
                plain = y.float() * torch.rsqrt(y.float().square().mean(1, keepdim=True) + 1e-6) \
                    * w[:, None]
                assert torch.equal(out[2, :, T // 2].isnan(), plain[2, :, T // 2].isnan())
                out8, scale, _ = rl.rms_norm_8bit(y, w, lengths=lengths)
                assert bool(out8[2, :, T // 2].float().isnan().all()) and scale[2, T // 2].isnan()
                keep = torch.ones(4, T, dtype=torch.bool, device="cuda")
                keep[2, T // 2] = False
                keep = keep[:, None].expand(4, D, T)
                assert torch.equal(out[keep], want[0][keep])
                assert torch.equal(out8.float()[keep], want[1].float()[keep])


def test_norm_gradients_against_differences(gpu_device):
    g = gen(3)
    x, w, go = normal(g, 2, 5, 7), normal(g, 5), normal(g, 2, 5, 7)
    grads = rl.rms_norm_backward(go, x, w)

    def loss(x, w):
        return float((ref.rms_norm(x, w)["out"][0] * go.cpu()).sum())

    x64, w64 = x.double(), w.double()
    for name, v in (("x", x64), ("weight", w64)):
        step = normal(g, *v.shape).double()
        up = (x64 + 1e-5 * step, w64) if name == "x" else (x64, w64 + 1e-5 * step)
        down = (x64 - 1e-5 * step, w64) if name == "x" else (x64, w64 - 1e-5 * step)
        slope = (loss(*up) - loss(*down)) / 2e-5
        got = getattr(grads, name).double()
        assert abs(float((got * step).sum()) - slope) <= 1e-5 * (float((got * step).abs().sum()) + 1)


def test_norm_captured_and_streams(gpu_device):
    g = gen(4)
    cases = [(normal(g, 3, 300, 130, dtype=torch.bfloat16), normal(g, 300)),
             (normal(g, 300, 5000), normal(g, 5000))]

    def both():
        got = []
        for x, w in cases:
            out, s = rl.rms_norm(x, w, x)
            got += [out, s, *rl.rms_norm_8bit(x, w)[:2], *rl.rms_norm_backward(out, s, w)]
        return got

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
            assert torch.equal(p.float(), w.float()) and torch.equal(q.float(), w.float())
