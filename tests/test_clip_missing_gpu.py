"""clip_grad_norm of a model some of whose parameters have no gradient."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_readme_example_gpu import readme_block, readme_names
from .test_sequence_gpu import gen

pytestmark = pytest.mark.gpu


def test_readme_clipping(gpu_device):
    """A model with a parameter that has no gradient."""
    names = readme_names(gen(91))
    block = readme_block("clip_grad_norm")
    exec(block[block.index("norm = "):], names)
    assert names["norm"].item() == pytest.approx(15 ** 0.5, rel=1e-12)
    assert names["model"].bias.grad is None


def test_clip_skips_missing_gradients(gpu_device):
    a, b = torch.ones(4, device="cuda"), torch.full((5,), 2.0, device="cuda")
    outs = [torch.empty_like(a), None, torch.empty_like(b)]
    assert rl.clip_grad_norm([a, None, b], 1.0, out=outs).item() == pytest.approx(24 ** 0.5)
    assert torch.allclose(outs[2], b / 24 ** 0.5)
    assert rl.clip_grad_norm([None, a], 1.0).item() == pytest.approx(2.0)
    with pytest.raises(ValueError):
        rl.clip_grad_norm([None, None], 1.0)
    with pytest.raises(ValueError):
        rl.clip_grad_norm([a, None], 1.0, out=[a.clone(), b.clone()])
