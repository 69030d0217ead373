"""A beam search's selection and reordering against plain forms in 64 bits and on the
host: which candidates are chosen, in which order, equal ones, beams that are finished
or not in use, tokens that are not allowed, infinities and NaN, and where every state
is afterwards."""
import math

import numpy as np
import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from .test_sequence_gpu import DTYPES, NAMES, gen, normal

pytestmark = pytest.mark.gpu

INF = float("inf")


def reference(logits, scores, picks, finished=None, pad_token=0):
    """Totals in float64 on the host; NaN first, then the highest, then the lowest
    beam and token."""
    x, s = logits.detach().cpu().double().numpy(), scores.detach().cpu().double().numpy()
    N, K, V = x.shape
    out = []
    for n in range(N):
        total = np.empty((K, V))
        for b in range(K):
            score = np.nan if s[n, b] == np.inf else s[n, b]  # no log probability
            if finished is not None and bool(finished[n, b]):
                total[b] = -np.inf
                total[b, pad_token] = score
            elif s[n, b] == -np.inf:
                total[b] = -np.inf
            elif np.isnan(score) or np.isnan(x[n, b]).any() or (x[n, b] == np.inf).any():
                total[b] = np.nan
            elif (x[n, b] == -np.inf).all():
                total[b] = -np.inf
            else:
                m = x[n, b].max()
                # m first: where logits are near 1e38, m + log(sum) is m
                total[b] = s[n, b] + ((x[n, b] - m) - np.log(np.exp(x[n, b] - m).sum()))
        flat = total.reshape(-1)
        rank = np.where(np.isnan(flat), np.inf, flat)
        first = np.where(np.isnan(flat), 0, 1)
        order = np.lexsort((np.arange(K * V), -rank, first))[:picks]
        out.append((flat[order], order % V, order // V))
    return [np.stack([o[i] for o in out]) if N else np.empty((0, picks)) for i in range(3)]


def check(logits, scores, picks, **kw):
    want = reference(logits, scores, picks, **kw)
    got = rl.beam_select(logits, scores, picks=picks, **kw)
    assert [t.dtype for t in got] == [torch.float32, torch.int32, torch.int32]
    np.testing.assert_array_equal(got.parents.cpu().numpy(), want[2])
    np.testing.assert_array_equal(got.tokens.cpu().numpy(), want[1])
    # 1e-6 of the sums, and the rounding to float32
    np.testing.assert_allclose(got.scores.cpu().numpy(), want[0], rtol=2.0 ** -23, atol=1e-6)
    return got


def inputs(g, N, K, V, dtype):
    scores = -20 * torch.rand(N, K, generator=g, device="cuda")
    return normal(g, N, K, V, dtype=dtype, scale=3.0), scores


# both chunk sizes, one token to several chunks, odd sizes, all picks from one beam
SHAPES = [(1, 1, 1, 1), (2, 1, 7, 5), (3, 4, 1, 4), (1, 4, 33, 64), (2, 3, 300, 8), (1, 64, 5, 64),
          (1, 5, 2048, 10), (3, 8, 2049, 8), (1, 2, 32000, 64), (1, 4, 65537, 4),
          (70, 8, 8195, 16), (300, 2, 9000, 3)]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES)
def test_select(dtype, gpu_device):
    for N, K, V, picks in SHAPES:
        print(f"select {dtype} {N}x{K}x{V} picks {picks}", flush=True)
        g = gen(N + V)
        logits, scores = inputs(g, N, K, V, dtype)
        check(logits, scores, picks)
        finished = (torch.rand(N, K, generator=g, device="cuda") < 0.4).to(torch.uint8)
        scores = torch.where(torch.rand(N, K, generator=g, device="cuda") < 0.2, -INF, scores)
        check(logits, scores, picks, finished=finished, pad_token=V - 1)


def test_select_equal_ones(gpu_device):
    """Ties within a beam, between beams of equal rows, and of everything."""
    g = gen(1)
    for N, K, V, picks in ((2, 3, 70, 9), (1, 4, 20000, 64), (140, 8, 8195, 8)):
        few = torch.randint(0, 3, (N, K, V), generator=g, device="cuda").float()
        scores = torch.zeros(N, K, device="cuda")
        check(few, scores, picks)
        check(few[:, :1].expand(N, K, V), scores, picks)
        flat = torch.zeros(N, K, V, device="cuda", dtype=torch.bfloat16)
        flat[..., ::2] = -0.0
        check(flat, scores, picks)
        check(torch.full_like(flat, torch.finfo(torch.bfloat16).min), scores, picks)


def test_select_tokens_that_are_not_allowed(gpu_device):
    g = gen(2)
    for N, K, V, picks in ((2, 3, 70, 20), (1, 4, 20000, 64), (140, 8, 8195, 8)):
        logits, scores = inputs(g, N, K, V, torch.float32)
        for share in (0.5, 0.99, 1.0):
            m = torch.rand(N, K, V, generator=g, device="cuda") < share
            check(logits.masked_fill(m, -INF), scores, picks)
        low = logits.masked_fill(m, torch.finfo(torch.float32).min)
        check(low, scores, picks)
        none = logits.clone()
        none[:, 0] = -INF  # one beam has nothing to go on with
        check(none, scores, picks)
        check(none, torch.full_like(scores, -INF), picks)


def test_select_infinities_and_nans(gpu_device):
    g = gen(3)
    for N, K, V, picks in ((4, 3, 70, 6), (4, 3, 2, 5), (4, 2, 20000, 5)):
        logits, scores = inputs(g, N, K, V, torch.float32)
        for bad in (float("nan"), INF):
            x = logits.clone()
            x[1, 1, V // 2] = bad
            check(x, scores, picks)
            # what a beam that is not in use, or finished, holds does not count
            s = scores.clone()
            s[1, 1] = -INF
            check(x, s, picks)
            finished = torch.zeros(N, K, device="cuda", dtype=torch.bool)
            finished[1, 1] = True
            check(x, scores, picks, finished=finished, pad_token=1)
            s[1, 1], s[2, 0] = float("nan"), INF
            check(logits, s, picks)


def test_select_strided_and_other_streams(gpu_device):
    g = gen(4)
    wide = normal(g, 6, 10, 3007, dtype=torch.float16)
    scores = torch.zeros(3, 5, device="cuda")
    want = check(wide[::2, 1::2, 3:2999], scores, 7)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        rl.beam_select(wide[::2, 1::2, 3:2999], scores, picks=7)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = rl.beam_select(wide[::2, 1::2, 3:2999], scores, picks=7)
    torch.cuda.synchronize()
    for _ in range(3):
        got.tokens.zero_()
        graph.replay()
        eager = rl.beam_select(wide[::2, 1::2, 3:2999], scores, picks=7)
        torch.cuda.synchronize()
        for p, q, w in zip(got, eager, want):
            assert torch.equal(p, w) and torch.equal(q, w)
    assert rl.beam_select(wide[:0, :5], scores[:0]).tokens.shape == (0, 5)


# ----------------------------------------------------------------- the reordering
def reordered(pools, slots, parents):
    """Beam by beam on the host."""
    places = pools[0].shape[0] if pools else 0
    now = [p.clone() for p in pools]
    new = []
    for mine, chosen in zip(slots.tolist(), parents.tolist()):
        K = len(mine)
        free = [mine[p] for p in range(K) if p not in chosen]
        seen, row = set(), []
        for p in chosen:
            if 0 <= p < K and p not in seen:
                seen.add(p)
                row.append(mine[p])
                continue
            row.append(free.pop(0))
            if 0 <= p < K and 0 <= mine[p] < places and 0 <= row[-1] < places:
                for a, b in zip(now, pools):
                    a[row[-1]] = b[mine[p]]
        new.append(row)
    return now, torch.tensor(new, dtype=torch.int32).reshape(slots.shape)


def pools_of(g, places):
    """States of several types, with places of odd numbers of bytes."""
    return [normal(g, places, 37, 3, dtype=torch.bfloat16), normal(g, places, 1000),
            torch.randint(0, 256, (places, 13), generator=g, device="cuda").to(torch.uint8),
            normal(g, places, 5000, 2, dtype=torch.float16), normal(g, places, 1),
            normal(g, places, 0)]


@pytest.mark.parametrize("N,K", [(1, 1), (1, 2), (3, 4), (5, 64), (2, 63), (40, 7)])
def test_reorder(N, K, gpu_device):
    g = gen(N * K)
    places = N * K + 5
    pools = pools_of(g, places)
    slots = torch.randperm(places, generator=g, device="cuda")[:N * K].int().view(N, K)
    for parents in (torch.randint(0, K, (N, K), generator=g, device="cuda").int(),
                    torch.zeros(N, K, device="cuda").int(),
                    torch.arange(K, device="cuda").int().expand(N, K).contiguous(),
                    torch.arange(K, device="cuda").int().flip(0).expand(N, K).contiguous()):
        print(f"reorder {N}x{K}", flush=True)
        before = [p.clone() for p in pools]
        want, new = reordered(pools, slots, parents)
        versions = [p._version for p in pools]
        got = rl.beam_reorder(pools, slots, parents)
        assert torch.equal(got.cpu(), new)
        for p, w in zip(pools, want):
            assert torch.equal(p, w)
        assert all(p._version > v for p, v in zip(pools, versions))
        # every beam finds its parent's state
        for p, b in zip(pools, before):
            at = slots.long().gather(1, parents.long())
            assert torch.equal(p[got.long()], b[at])
        slots = got


def test_reorder_empty_seats_and_unused_beams(gpu_device):
    g = gen(9)
    pools = pools_of(g, 6)
    slots = torch.tensor([[0, -1, 2, 7], [5, 1, 3, 4]], device="cuda", dtype=torch.int32)
    for parents in ([[0, 0, 2, 2], [3, 3, -1, 0]], [[1, 1, 1, 0], [9, 9, 9, 9]],
                    [[3, 0, 0, 0], [2, 2, 5, 2]]):
        parents = torch.tensor(parents, device="cuda", dtype=torch.int32)
        want, new = reordered(pools, slots, parents)
        got = rl.beam_reorder(pools, slots, parents)
        assert torch.equal(got.cpu(), new)
        for p, w in zip(pools, want):
            assert torch.equal(p, w)


def test_reorder_many_pools(gpu_device):
    """More pools than a launch takes, none at all, and places without bytes."""
    g = gen(10)
    pools = [normal(g, 9, 1 + i % 7) for i in range(200)]
    slots = torch.tensor([[8, 3, 5], [0, 1, 2]], device="cuda", dtype=torch.int32)
    parents = torch.tensor([[2, 2, 2], [0, 1, 0]], device="cuda", dtype=torch.int32)
    want, new = reordered(pools, slots, parents)
    assert torch.equal(rl.beam_reorder(pools, slots, parents).cpu(), new)
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    assert torch.equal(rl.beam_reorder([], slots, parents).cpu(), new)
    empty = torch.zeros(0, 3, device="cuda")
    assert torch.equal(rl.beam_reorder([empty], slots, parents).cpu(), new)
    assert rl.beam_reorder(pools, slots[:0], parents[:0]).shape == (0, 3)


def test_reorder_large_places(gpu_device):
    """Offsets past 2^32 bytes."""
    pool = torch.empty(5, 300_000_011, dtype=torch.float32, device="cuda")
    pool.copy_(torch.arange(5, device="cuda", dtype=torch.float32)[:, None].expand_as(pool))
    slots = torch.tensor([[4, 0, 3, 1]], device="cuda", dtype=torch.int32)
    got = rl.beam_reorder([pool], slots, torch.tensor([[2, 2, 0, 2]], device="cuda").int())
    assert got.tolist() == [[3, 0, 4, 1]]
    for place, value in enumerate((3, 3, 2, 3, 4)):
        assert bool((pool[place] == value).all())


def test_reorder_captured(gpu_device):
    g = gen(11)
    pools = pools_of(g, 9)
    start = [p.clone() for p in pools]
    slots = torch.tensor([[8, 3, 5], [0, 1, 2]], device="cuda", dtype=torch.int32)
    parents = torch.tensor([[2, 2, 2], [0, 1, 0]], device="cuda", dtype=torch.int32)
    want, new = reordered(pools, slots, parents)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        rl.beam_reorder(pools, slots, parents)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = rl.beam_reorder(pools, slots, parents)
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(pools, start):
            p.copy_(s)
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), new)
        for p, w in zip(pools, want):
            assert torch.equal(p, w)


def test_math_of_a_search(gpu_device):
    """A whole search over a fixed table of log probabilities finds its best sequences."""
    g = gen(12)
    V, K, steps = 6, 36, 3
    table = torch.log_softmax(normal(g, V, V, scale=2.0), 1)
    scores = torch.full((1, K), -INF, device="cuda")
    scores[0, 0] = 0.0
    state = torch.zeros(K, 1, device="cuda", dtype=torch.int64)  # the last token
    trace = torch.zeros(K, steps, device="cuda", dtype=torch.int64)
    slots = torch.arange(K, device="cuda", dtype=torch.int32)[None]
    for i in range(steps):
        at = slots[0].long()
        choice = rl.beam_select(table[state[at, 0]][None], scores)
        slots = rl.beam_reorder([state, trace], slots, choice.parents)
        at = slots[0].long()
        state[at, 0] = choice.tokens[0].long()
        trace[at, i] = choice.tokens[0].long()
        scores = choice.scores
    every = [(float(table[0, a] + table[a, b] + table[b, c]), (a, b, c))
             for a in range(V) for b in range(V) for c in range(V)]
    every.sort(key=lambda e: -e[0])
    # 36 beams hold all prefixes of two tokens, so the search is exhaustive
    found = trace[slots[0].long()].tolist()
    for k in range(K):
        assert math.isclose(float(scores[0, k]), every[k][0], abs_tol=1e-5)
        assert tuple(found[k]) == every[k][1]
