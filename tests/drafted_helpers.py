"""Inputs and comparisons of the tests of drafted tokens over the paged cache."""
from __future__ import annotations

import random

import torch

from paged_helpers import HALF

# What a weight loses where it is rounded to the operands' type for the product with the values:
# half a step, relative to the weight.
WEIGHT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def random_trees(batch, tokens, seed=0):
    """Masks [batch][tokens] of random trees, as non-negative ints."""
    rng = random.Random(seed)
    out = []
    for _ in range(batch):
        m = []
        for t in range(tokens):
            p = rng.randint(max(-1, t - 4), t - 1)
            m.append((m[p] if p >= 0 else 0) | 1 << t)
        out.append(m)
    return out


def as_tensor(masks):
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in line] for line in masks],
                        dtype=torch.int64)


def check_tree(o, lse, want_o, want_lse, magnitude, what="", grow=1.0):
    """o against the 64-bit result: half a step of its type for the output's rounding; WEIGHT of
    sum_j p_j |v_j| for the weights' rounding; and 2^-12 of that sum for the scores and the total
    (the arithmetic is in paged_helpers.check_attention), times `grow` where scores are so many
    times larger than the inputs assumed there.  The LSE as there."""
    half, weight = HALF[o.dtype], WEIGHT[o.dtype] + grow * 2.0 ** -12
    o, lse = o.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isnan(o), torch.isnan(want_o)), what
    assert torch.equal(torch.isnan(lse), torch.isnan(want_lse)), what
    inf = torch.isinf(want_o)
    assert torch.equal(o[inf], want_o[inf]), what
    fine = torch.isfinite(want_o)
    least = 2.0 ** -25 if half == HALF[torch.float16] else 0.0  # half of fp16's least step
    off = (o - want_o).abs()[fine]
    allowed = (half * want_o.abs() + weight * magnitude + least)[fine] + 1e-30
    worst = (off / allowed).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: o off by {worst:.3g} of what rounding allows"
    inf = torch.isinf(want_lse)
    assert torch.equal(lse[inf], want_lse[inf]), what
    fine = torch.isfinite(want_lse)
    off = ((lse - want_lse).abs() - 2.0 ** -21 * want_lse.abs())[fine]
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= grow * 1e-4, f"{what}: lse off by {worst:.3g}"


def angle_table(positions, dim, base=10000.0):
    """fp32 [positions, dim]: cosines, then sines, of the usual angles."""
    f = base ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()
