"""README's example of a residual block and of a search runs, and gives what the calls'
references give."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from . import blocks_reference as ref
from .test_beams_gpu import reference, reordered
from .test_readme_example_gpu import readme_block
from .test_sequence_gpu import check, gen, normal

pytestmark = pytest.mark.gpu


def test_readme_block(gpu_device):
    g = gen(3)
    N, ch, T, K, V = 3, 20, 40, 2, 50
    names = dict(rl=rl, decay=normal(g, ch) - 3, weight=normal(g, ch), h0=normal(g, N, ch),
                 starts=(torch.rand(N, T, generator=g, device="cuda") < 0.2).to(torch.uint8),
                 slots=torch.arange(N * K, device="cuda", dtype=torch.int32).view(N, K),
                 pool=normal(g, N * K + 2, ch), conv_pool=normal(g, N * K + 2, ch, 3),
                 logits=normal(g, N, K, V), scores=normal(g, N, K),
                 done=torch.zeros(N, K, device="cuda", dtype=torch.uint8))
    for k in ("new", "s", "x", "input_gate", "decay_gate", "grad_h", "grad_y", "grad_s"):
        names[k] = normal(g, N, ch, T)
    for k in ("x_t", "i_t", "r_t"):
        names[k] = normal(g, N * K, ch)
    given = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in names.items()}
    exec(readme_block("gated_recurrence_backward"), names)
    normed = ref.rms_norm(given["new"], given["weight"], given["s"], grad_out=given["grad_y"],
                          grad_sum=given["grad_s"])
    check(names["y"], normed["out"], "y")
    check(names["gn"].x, normed["x"], "norm's gradient")
    check(names["gn"].weight, normed["weight"], "norm's weight")
    want = ref.gated(given["x"], given["input_gate"], given["decay_gate"], given["decay"],
                     state=given["h0"], flags=given["starts"], grad_out=given["grad_h"])
    check(names["last"], want["final"], "last")
    for k in ("x", "input_gate", "decay_gate", "decay", "state"):
        check(getattr(names["g"], k), want[k], k)
    step = ref.gated(*(given[k][:, :, None] for k in ("x_t", "i_t", "r_t")), given["decay"],
                     state=given["pool"][:N * K])
    check(names["h"][:, :, None], step["out"], "step")
    best = reference(given["logits"], given["scores"], K)
    assert names["best"].tokens.cpu().numpy().tolist() == best[1].tolist()
    stepped = given["pool"].clone()
    stepped[:N * K] = names["h"]
    pools, slots = reordered([stepped, given["conv_pool"]], given["slots"], names["best"].parents)
    assert torch.equal(names["slots"].cpu(), slots)
    assert torch.equal(names["pool"], pools[0]) and torch.equal(names["conv_pool"], pools[1])
