"""clip_grad_norm against sums in 64 bits: the norm to 1e-12 relative (fp64
squares and sums of at most 10^7 terms: 10^7 * 2^-53 is 1.1e-9 at worst, and
each workgroup's sums are far shorter; 1e-10 is asked), scaled values to the
scale's and the product's roundings and one to their type."""
import math

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import sequence_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check(grads, max_norm, eps=1e-6, **kw):
    norm, scaled = ref.clip(grads, max_norm, eps)
    before = [t.clone() for t in grads]
    got = rl.clip_grad_norm(grads, max_norm, eps, **kw)
    assert got.shape == (1,) and got.dtype == torch.float64
    assert got.item() == pytest.approx(norm, rel=1e-10, abs=0)
    outs = kw.get("out") or grads
    for i, (o, (value, bound)) in enumerate(zip(outs, scaled)):
        tol = ref.tolerance(value, bound, o.dtype)
        assert bool(((o.cpu().double() - value).abs() <= tol).all()), f"tensor {i}"
    if "out" in kw:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    return got


SIZES = [[1], [15, 16, 17], [4095, 4096, 4097], [1 << 20], [3] * 95, [5] * 96, [7] * 97,
         [2] * 300 + [100_001], [8_400_000, 1, 0, 12]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", DTYPES + ["mixed"], ids=["f32", "bf16", "f16", "mixed"])
def test_clip(dtype, sizes, gpu_device):
    g = torch.Generator(device="cuda").manual_seed(len(sizes))
    total = math.sqrt(sum(sizes))
    for max_norm in (0.3 * total, 1e6, 0.0):
        grads = [normal(g, n, dtype=DTYPES[i % 3] if dtype == "mixed" else dtype)
                 for i, n in enumerate(sizes)]
        print(f"clip {dtype} {len(sizes)} tensors to {max_norm}", flush=True)
        check(grads, max_norm, out=[torch.full_like(t, 9.0) for t in grads])
        check(grads, max_norm)


def test_layouts_and_alignment(gpu_device):
    g = torch.Generator(device="cuda").manual_seed(1)
    for dtype in DTYPES:
        base = normal(g, 5000, dtype=dtype)
        grads = [base[1:1001], base[1001:1020].view(19), base[2003:4003].view(40, 50).t(),
                 normal(g, 2, 3, 4, 5, dtype=dtype).to(memory_format=torch.channels_last),
                 normal(g, dtype=dtype)]
        around = base.clone()
        check(grads, 1.0)
        keep = torch.ones(5000, dtype=torch.bool, device="cuda")
        keep[1:1020] = False
        keep[2003:4003] = False
        assert torch.equal(base[keep], around[keep])
        with pytest.raises(ValueError):
            rl.clip_grad_norm([base[::2]], 1.0)


def test_norm_only(gpu_device):
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [normal(g, 1000), normal(g, 10, dtype=torch.float16)]
    before = [t.clone() for t in grads]
    n = rl.clip_grad_norm(grads, math.inf)
    assert n.item() == pytest.approx(ref.clip(grads, math.inf, 0)[0], rel=1e-10)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert rl.clip_grad_norm([torch.empty(0, device="cuda")], 1.0).item() == 0.0


def test_large_and_small_values(gpu_device):
    """Squares past float32's range on both sides."""
    for v in (3e30, 1e-30):
        t = torch.full((1000,), v, device="cuda")
        n = rl.clip_grad_norm([t], math.inf)
        assert n.item() == pytest.approx(float(t[0]) * math.sqrt(1000), rel=1e-10)
    t = torch.full((1000,), 3e30, device="cuda")
    rl.clip_grad_norm([t], 1.0)
    assert torch.allclose(t, torch.full_like(t, 1 / math.sqrt(1000)), rtol=1e-6)


def test_nonfinite(gpu_device):
    nan = torch.ones(10, device="cuda")
    nan[3] = math.nan
    n = rl.clip_grad_norm([nan, torch.ones(5, device="cuda")], 1.0)
    assert math.isnan(n.item()) and nan.isnan().all()
    inf = torch.ones(10, device="cuda")
    inf[3] = -math.inf
    n = rl.clip_grad_norm([inf], 1.0)
    assert math.isinf(n.item()) and inf[3].isnan() and not inf[:3].any()
    zero = torch.zeros(10, device="cuda")
    assert rl.clip_grad_norm([zero], 0.0, eps=0.0).item() == 0.0 and not zero.any()


def test_repeatable(gpu_device):
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [normal(g, n) for n in (100_000, 33, 1_000_000, 7)]
    a = rl.clip_grad_norm(grads, math.inf)
    for _ in range(3):
        assert torch.equal(a, rl.clip_grad_norm(grads, math.inf))


def test_refusals(gpu_device):
    t = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        rl.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        rl.clip_grad_norm([t.cpu()], 1.0)
    with pytest.raises(ValueError):
        rl.clip_grad_norm([t, t.cpu()], 1.0)
    with pytest.raises(TypeError):
        rl.clip_grad_norm([t.double()], 1.0)
    with pytest.raises(ValueError):
        rl.clip_grad_norm([t], 1.0, out=[])
    with pytest.raises(ValueError):
        rl.clip_grad_norm([t], 1.0, out=[t.half()])
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(max_norm=1.0, eps=-1.0)):
        with pytest.raises(rl.RlcaError):
            rl.clip_grad_norm([t], **kw)
    with pytest.raises(rl.RlcaError):
        rl.clip_grad_norm([t, t], 1.0)


def test_first_call_on_a_stream_is_captured(gpu_device):
    """No eager call has made the stream's workspace: a captured call brings its
    own, and eager calls on that stream before and between replays are right."""
    g = torch.Generator(device="cuda").manual_seed(5)
    new = [[normal(g, n) for n in (70_001, 5, 4096)] for _ in range(4)]
    grads, outs = [t.clone() for t in new[0]], [torch.empty_like(t) for t in new[0]]
    rl.clip_grad_norm(grads, 1.0, out=outs)  # on another stream, which loads the kernels
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        norm = rl.clip_grad_norm(grads, 1.0, out=outs)
    for values in new:
        with torch.cuda.stream(stream):
            eager_out = [torch.empty_like(t) for t in values]
            eager = rl.clip_grad_norm(values, 1.0, out=eager_out)
        stream.synchronize()
        for t, v in zip(grads, values):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want, scaled = ref.clip(values, 1.0, 1e-6)
        assert eager.item() == pytest.approx(want, rel=1e-10, abs=0)
        assert norm.item() == eager.item()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager_out))
