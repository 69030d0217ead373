"""The order of a beam search's candidates whose totals float64 does not tell apart: the
lower beam first, and of one beam's the higher logit, then the lower token, whatever
the sizes that the call's launch depends on."""
import math

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_sequence_gpu import gen, normal

pytestmark = pytest.mark.gpu


def expected(logits, scores, picks):
    """Python's sort of one search's candidates, the totals in float64."""
    x, s = logits.double().cpu().tolist(), scores.double().cpu().tolist()
    every = []
    for b, (row, score) in enumerate(zip(x, s)):
        m = max(row)
        lse = math.log(sum(math.exp(v - m) for v in row))
        # a token that is not allowed ranks last, by beam and token
        every += [(-(score - lse + (v - m)), b, -v, t) if v > -math.inf else (math.inf, b, 0, t)
                  for t, v in enumerate(row)]
    every.sort()
    return [(b, t) for _, b, _, t in every[:picks]]


def chosen(choice, n):
    return list(zip(choice.parents[n].tolist(), choice.tokens[n].tolist()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("K,V,picks", [(1, 50, 4), (3, 2500, 7), (2, 9000, 64), (1, 14000, 1)])
def test_order_of_totals_that_round_to_one(K, V, picks, dtype, gpu_device):
    g = gen(V)
    logits = normal(g, 1, K, V, dtype=dtype, scale=3.0)
    huge = logits.clone()
    huge[:, :, V // 2] = 1e30  # the others' totals are -1e30 all
    tiny = (logits.float() * 1e-20).to(dtype)
    unused = torch.full((1, K), -1e30, device="cuda")
    lowest = torch.full((1, K), torch.finfo(torch.float32).min, device="cuda")
    zero = torch.zeros(1, K, device="cuda")
    masked = logits.masked_fill(torch.rand(1, K, V, generator=g, device="cuda") < 0.5, -math.inf)
    first = unused.clone()
    first[0, 0] = 0.0
    few = masked.clone()
    few[0, 0, 2:] = -math.inf  # less than `picks` from the first beam
    for name, x, s in (("unused", logits, unused), ("lowest", logits, lowest),
                       ("masked", masked, unused), ("few", few, first), ("huge", huge, zero),
                       ("tiny", tiny, zero)):
        print(f"order {name} {dtype} {K}x{V} picks {picks}", flush=True)
        want = expected(x[0], s[0], picks)
        # alone, and among as many searches as make the launch take larger chunks
        for N in (1, 160):
            got = rl.beam_select(x.expand(N, K, V), s.expand(N, K).contiguous(), picks=picks)
            assert chosen(got, 0) == want
            assert chosen(got, N - 1) == want
