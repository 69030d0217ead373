"""causal_conv_step at channel counts whose channels * taps pass 2^31."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W,D", [(4, (1 << 31) // 3 + 40), (4, (1 << 30)), (3, (1 << 30) + 17)],
                         ids=["4x715827922", "4x1073741824", "3x1073741841"])
def test_conv_step_of_many_channels(W, D, gpu_device):
    """All channels alike but some, spread over the range: every output and
    state of the first kind equal, the others' by the formula.  (channels *
    (W - 1) states pass 2^31 in all three.)"""
    print(f"conv step W={W} channels={D}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(W)
    weight = torch.full((D, W), 0.5, device="cuda")
    state = torch.full((1, D, W - 1), 0.25, device="cuda", dtype=torch.bfloat16)
    x = torch.full((1, D), 2.0, device="cuda", dtype=torch.bfloat16)
    at = torch.cat([torch.arange(12, device="cuda"), torch.arange(D - 12, D, device="cuda"),
                    torch.randint(12, D - 12, (300,), generator=g, device="cuda")]).unique()
    weight[at] = torch.randn(len(at), W, generator=g, device="cuda")
    state[0, at] = torch.randn(len(at), W - 1, generator=g, device="cuda").to(torch.bfloat16)
    x[0, at] = torch.randn(len(at), generator=g, device="cuda").to(torch.bfloat16)
    old, new = state[0, at].clone(), x[0, at].clone()
    out = rl.causal_conv_step(x, weight, None, state, silu=False)
    taps = torch.cat([old, new[:, None]], 1)
    want = (taps.double() * weight[at].double()).sum(1)
    mag = (taps.double() * weight[at].double()).abs().sum(1)
    # W products and sums in fp32, one rounding to bf16
    tol = (W + 2) * 2.0 ** -24 * mag + 2.0 ** -8 * (want.abs() + mag * 2.0 ** -20)
    assert bool(((out[0, at].double() - want).abs() <= tol).all())
    assert torch.equal(state[0, at], taps[:, 1:])
    common = 0.5 * 2.0 + 0.5 * 0.25 * (W - 1)  # exact in bf16
    out[0, at] = common
    assert bool((out == common).all())
    state[0, at] = torch.tensor([0.25] * (W - 2) + [2.0], device="cuda", dtype=torch.bfloat16)
    for j in range(W - 1):
        assert bool((state[0, :, j] == (2.0 if j == W - 2 else 0.25)).all()), j
