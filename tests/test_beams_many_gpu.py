"""A beam search's calls at their largest counts: more searches than a launch has rows of
workgroups, and a vocabulary of many chunks a beam."""
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_beams_gpu import check
from .test_sequence_gpu import gen, normal

pytestmark = pytest.mark.gpu


def test_many_searches(gpu_device):
    """70001 searches of 2 beams: chosen, then their states moved, against sorted totals in
    float64 (where no two that matter are within 2e-6) and indexed states."""
    g = gen(1)
    N, K, V = 70001, 2, 5
    logits = normal(g, N, K, V, scale=3.0)
    scores = -20 * torch.rand(N, K, generator=g, device="cuda")
    total = (scores.double()[:, :, None] + logits.double().log_softmax(2)).view(N, K * V)
    want, index = total.sort(dim=1, descending=True, stable=True)
    clear = (want[:, :K] - want[:, 1:K + 1]).amin(1) > 2e-6
    assert clear.float().mean() > 0.999
    got = rl.beam_select(logits, scores)
    flat = got.parents.long() * V + got.tokens.long()
    assert torch.equal(flat[clear], index[:, :K][clear])
    assert ((got.scores.double() - want[:, :K]).abs() <= 2e-6 + want[:, :K].abs() * 2.0 ** -24).all()

    places = N * K + 9
    pool = normal(g, places, 3)
    before = pool.clone()
    slots = torch.randperm(places, generator=g, device="cuda")[:N * K].int().view(N, K)
    new = rl.beam_reorder([pool], slots, got.parents)
    # each beam finds its parent's state, all at places of their own among the search's
    at = slots.long().gather(1, got.parents.long())
    assert torch.equal(pool[new.long()], before[at])
    assert torch.equal(new.sort(dim=1).values, slots.sort(dim=1).values)
    others = torch.ones(places, dtype=torch.bool, device="cuda")
    others[slots.long().view(-1)] = False
    assert torch.equal(pool[others], before[others])


@pytest.mark.parametrize("picks", [1, 64])
def test_a_large_vocabulary(picks, gpu_device):
    g = gen(2)
    for dtype in (torch.float16, torch.float32):
        logits = normal(g, 1, 1, 5_000_003, dtype=dtype, scale=3.0)
        check(logits, torch.full((1, 1), -3.0, device="cuda"), picks)
