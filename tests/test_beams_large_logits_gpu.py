"""A beam search's selection over logits of any finite size: tokens masked by a large
finite number, in scattered places, in runs that fill whole threads and chunks, and
everywhere; large logits of either sign; and values on both sides of where the sums'
arithmetic changes.  Against the 64-bit form on the host."""
import random

import pytest
import torch

from .test_beams_gpu import check, inputs
from .test_sequence_gpu import gen, normal

pytestmark = pytest.mark.gpu

# one chunk a beam, several of the smaller kind, several of the larger kind
SHAPES = [(2, 3, 70, 9), (1, 4, 20000, 7), (140, 8, 8195, 8)]
FILLS = [-1e4, -4194303.0, -4194304.0, -4.2e6, -1.7e7, -1e9, -1e10, -1e20, -1e30, -1e36, -3e38]


def masks(g, N, K, V):
    """Places to fill: scattered ones, a run to the end, a run in the middle, all of one
    beam, all but two tokens, and all."""
    at = torch.arange(V, device="cuda").expand(N, K, V)
    yield torch.rand(N, K, V, generator=g, device="cuda") < 0.7
    yield at >= V // 3
    yield (at >= V // 5) & (at < V - V // 7)
    yield (torch.arange(K, device="cuda") == K // 2)[None, :, None].expand(N, K, V)
    yield (at != V // 2) & (at != V - 1)
    yield at >= 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fill", FILLS)
def test_select_with_a_finite_mask(fill, dtype, gpu_device):
    for N, K, V, picks in SHAPES:
        print(f"select {dtype} {N}x{K}x{V} picks {picks} fill {fill}", flush=True)
        g = gen(N + V)
        logits, scores = inputs(g, N, K, V, dtype)
        for m in masks(g, N, K, V):
            check(logits.masked_fill(m, fill), scores, picks)


def test_select_with_a_finite_mask_in_fp16(gpu_device):
    for N, K, V, picks in SHAPES:
        g = gen(N + V)
        logits, scores = inputs(g, N, K, V, torch.float16)
        for fill in (-1e4, torch.finfo(torch.float16).min):
            for m in masks(g, N, K, V):
                check(logits.masked_fill(m, fill), scores, picks)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [1e7, 1e10, 1e20, 1e36, 3e38])
def test_select_of_large_logits(size, dtype, gpu_device):
    for N, K, V, picks in SHAPES:
        print(f"select {dtype} {N}x{K}x{V} picks {picks} size {size}", flush=True)
        g = gen(N + V)
        logits, scores = inputs(g, N, K, V, dtype)
        one = logits.clone()
        one[:, :, V // 3] = size
        check(one, scores, 1)
        check(torch.full_like(logits, size), scores, picks)
        check((logits / logits.abs().max() * size).to(dtype), scores, 1)


def test_select_around_the_change(gpu_device):
    """Logits a few units apart, about +-2^22 and far from it: log probabilities as
    exact there as near 0."""
    g = gen(5)
    for N, K, V, picks in SHAPES:
        for about in (0.0, 1e3, 4194300.0, -4194300.0, 4194304.0, -4194304.0, 5e6, -5e6, 8e6):
            # as they are rounded there; equal ones are many
            x = about + (normal(g, N, K, V) * 8).round() / 4
            scores = -20 * torch.rand(N, K, generator=g, device="cuda")
            check(x, scores, picks)


@pytest.mark.parametrize("seed", range(12))
def test_select_random_masks(seed, gpu_device):
    r = random.Random(seed)
    g = gen(300 + seed)
    K, V = r.choice([1, 2, 5, 8]), int(2 ** r.uniform(1, 15))
    N = r.randint(1, max(1, min(80, 800_000 // (K * V))))
    picks = min(64, K * V, r.choice([1, K, 2 * K]))
    dtype = r.choice([torch.float32, torch.bfloat16])
    fill = r.choice([-1, -1, 1]) * r.choice([1e5, 3e6, 5e6, 1e8, 1e10, 1e22, 1e30, 1e37])
    share = r.choice([0.05, 0.5, 0.95, 0.999])
    if fill > 0:  # below such a logit float64 no longer tells the others' totals apart
        picks = 1
    print(f"select {dtype} {N}x{K}x{V} picks {picks} fill {fill} share {share}", flush=True)
    logits, scores = inputs(g, N, K, V, dtype)
    at = torch.rand(N, K, V, generator=g, device="cuda") < share
    if r.random() < 0.5:  # runs of 24, a thread's
        at = at[:, :, ::24].repeat_interleave(24, 2)[:, :, :V]
    check(logits.masked_fill(at, fill), scores, picks)
