"""README's example of a model core: its gradients are those of its forward calls."""
import os
import re

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import sequence_reference as ref
from .test_sequence_gpu import check, gen, normal, scan_inputs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_block(word):
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if word in b)


def readme_names(g):
    """The names that README's model core takes as given."""
    N, ch, S, T = 3, 20, 4, 9
    t = scan_inputs(g, N, ch, S, T, 1, torch.float32, True)
    names = {k: v for k, v in t.items() if k != "u"}
    names.update(rl=rl, x=normal(g, N, ch, T), weight=normal(g, ch, 4), bias=normal(g, ch),
                 conv_state=normal(g, N, ch, 3), conv0=normal(g, N, ch, 3),
                 h0=normal(g, N, ch, S), grad_y=normal(g, N, ch, T),
                 starts=(torch.rand(N, T, generator=g, device="cuda") < 0.2).to(torch.uint8),
                 slots=torch.arange(N, device="cuda").int(), conv_pool=normal(g, N + 2, ch, 3),
                 scan_pool=normal(g, N + 2, ch, S), x_t=normal(g, N, ch))
    for k in ("delta", "B", "C", "z"):
        names[k + "_t"] = t[k][..., 0].contiguous()
    names["model"] = torch.nn.Linear(5, 3).cuda()
    names["model"].weight.grad = torch.ones(3, 5, device="cuda")  # the bias has none
    return names


def test_readme_gradients(gpu_device):
    """The example's convolution gradients are those of its forward call, with
    the state that the row began from."""
    names = readme_names(gen(90))
    given = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in names.items()}
    block = readme_block("causal_conv_backward")
    exec(block[:block.index("norm = ")], names)
    state = given["conv0" if "conv0" in block else "conv_state"]
    want = ref.conv(given["x"], given["weight"], given["bias"], state, given["starts"],
                    grad_out=names["g"].u)
    for name in ("x", "weight", "bias", "state"):
        check(getattr(names["gc"], name), want[name], name)
