"""The norm's 8-bit output where its values lie near the least scale of 2^-120 or the
factor that makes 8-bit values of the inputs leaves float32's range: tiny inputs, tiny
weights, the smallest eps, and weights of 0 beside one large channel.  Against the
64-bit reference, in rows over time and in dense rows of channels."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import blocks_reference as ref
from .test_sequence_gpu import check, gen, normal

pytestmark = pytest.mark.gpu

# threads of 256, 512 and 1024, channels that are read twice, a wave and a workgroup a row
SHAPES = [(3, 70, 9), (2, 300, 33), (2, 1100, 20), (1, 2500, 70), (5, 64, 1), (3, 2500, 1),
          (2, 9000, 1)]


def check_8bit(x, w, res=None, eps=ref.EPS, lengths=None):
    want = ref.rms_norm(x, w, res, eps=eps, lengths=lengths)
    q, scale, _ = rl.rms_norm_8bit(x, w, res, eps=eps, lengths=lengths)
    check(scale, want["scale"], "scale")
    check(q.cpu().double() * scale.cpu().double().unsqueeze(1), want["dequantized"], "8 bits")
    check(rl.rms_norm(x, w, res, eps=eps, lengths=lengths)[0], want["out"], "out")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size,weight,eps", [
    # by eps 1e-6 a root of 1e-3: outputs about 1e-31 .. 1e-34, on both sides of 448 / 2^120
    (1e-34, 1.0, 1e-6), (1e-36, 1.0, 1e-6), (1e-37, 1.0, 1e-6),
    (1.0, 1e-30, 1e-6), (1.0, 1e-33, 1e-6), (1.0, 1e-35, 1e-6), (1e-3, 1e-33, 1e-6),
    (1e10, 1e-34, 1e-6), (1e30, 1e-34, 1e-6), (1e30, 1e-37, 1e-6),
    # by eps 1e-30 a root of 1e-15: outputs of ordinary size from tiny inputs
    (1e-20, 1.0, 1e-30), (1e-30, 1.0, 1e-30), (1e-36, 1.0, 1e-30), (1e-30, 1e-20, 1e-30),
])
def test_8bit_of_small_values(size, weight, eps, dtype, gpu_device):
    for N, D, T in SHAPES:
        g = gen(D + T)
        print(f"8 bit {dtype} {N}x{D}x{T} size {size} weight {weight} eps {eps}", flush=True)
        # one step in two is ordinary, and one sequence; magnitudes within a factor of 100,
        # so that all products stay normal numbers
        x = torch.rand(N, D, T, generator=g, device="cuda") + 0.01
        x *= torch.where(torch.rand(N, D, T, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        x[:, :, ::2] *= size
        w = weight * (0.5 + torch.rand(D, generator=g, device="cuda"))
        x = x.to(dtype)
        res = torch.zeros_like(x)
        lengths = torch.full((N,), T, device="cuda", dtype=torch.int32)
        lengths[0] = T - 1
        check_8bit(x, w, eps=eps)
        check_8bit(x, w, res, eps=eps, lengths=lengths)


def test_8bit_of_weights_that_are_0(gpu_device):
    """A channel far above the root mean square, where the weights are 0: 0, not NaN."""
    for dtype in (torch.float32, torch.bfloat16):
        for T in (1, 9):
            x = torch.zeros(2, 70001, T, device="cuda", dtype=dtype)
            x[:, 5] = 1e4
            for w in (torch.zeros(70001, device="cuda"), torch.full((70001,), 1e-38, device="cuda")):
                q, scale, _ = rl.rms_norm_8bit(x, w)
                want = ref.rms_norm(x, w)
                check(scale, want["scale"], "scale")
                check(q.cpu().double() * scale.cpu().double().unsqueeze(1), want["dequantized"],
                      "8 bits")


def test_8bit_of_ordinary_values_beside_zeros(gpu_device):
    """Steps of zeros, padded ones, beside others: scale 2^-120 and 0, the others as alone."""
    g = gen(3)
    for N, D, T in SHAPES:
        x = normal(g, N, D, T, dtype=torch.bfloat16)
        q, scale, _ = rl.rms_norm_8bit(x)
        y = x.clone()
        y[:, :, ::3] = 0
        q0, scale0, _ = rl.rms_norm_8bit(y)
        assert not q0[:, :, ::3].float().any() and bool((scale0[:, ::3] == 2.0 ** -120).all())
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[::3] = False
        assert torch.equal(q0.float()[:, :, keep], q.float()[:, :, keep])
        assert torch.equal(scale0[:, keep], scale[:, keep])
