"""What the recurrent policy's autograd functions pass on."""
import pytest
import torch

from linear_recurrence_scan_row_amd import recurrent_policy as rp
from . import sequence_reference as ref
from .test_sequence_gpu import check, gen, normal, scan_inputs

pytestmark = pytest.mark.gpu


def test_functions_pass_state_gradients(gpu_device):
    """States that require gradients get them, and B and C may have groups."""
    g = gen(92)
    N, ch, S, T, G = 3, 8, 5, 40, 2
    t = scan_inputs(g, N, ch, S, T, G, torch.float32, True)
    flags = (torch.rand(N, T, generator=g, device="cuda") < 0.05).to(torch.uint8)
    flags[:, 0] = 0
    go = normal(g, N, ch, T)
    h0, c0 = normal(g, N, ch, S), normal(g, N, ch, 3)
    order = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    leaves = [t[k].clone().requires_grad_() for k in order] + [h0.clone().requires_grad_()]
    rp._Scan.apply(*leaves, flags).backward(go)
    want = ref.scan(**t, state=h0, flags=flags, grad_y=go)
    for name, leaf in zip(order + ("state",), leaves):
        assert leaf.grad is not None, name
        check(leaf.grad, want[name], name)
    x, w, b = normal(g, N, ch, T), normal(g, ch, 4), normal(g, ch)
    leaves = [v.clone().requires_grad_() for v in (x, w, b, c0)]
    rp._Conv.apply(*leaves, flags).backward(go)
    want = ref.conv(x, w, b, c0, flags, grad_out=go)
    for name, leaf in zip(("x", "weight", "bias", "state"), leaves):
        assert leaf.grad is not None, name
        check(leaf.grad, want[name], name)


def test_no_second_derivative(gpu_device):
    """Refused, not silently left out."""
    g = gen(93)
    x, w, b = normal(g, 2, 4, 9), normal(g, 4, 3), normal(g, 4)
    x.requires_grad_()
    out = rp._Conv.apply(x, w, b, None, None)
    grad, = torch.autograd.grad(out.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (grad.sum() + x.sum()).backward()
    t = scan_inputs(g, 2, 4, 3, 9, 1, torch.float32, True)
    t = {k: v.requires_grad_() for k, v in t.items()}
    y = rp._Scan.apply(*(t[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")),
                       None, None)
    grad, = torch.autograd.grad(y.square().sum(), t["u"], create_graph=True)
    with pytest.raises(RuntimeError):
        (grad.sum() + t["u"].sum()).backward()
