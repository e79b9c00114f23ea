"""Plain implementations, in 64 bits on the CPU, of the operators of a step of drafted tokens over
the paged cache and of windowed attention: loops, straight from the definitions."""
from __future__ import annotations

import math

import torch

import paged_reference as ref


def rotate(x, cos_sin, positions, sections, interleaved):
    """x [T, heads, d] fp64; positions: for each axis a list of T; -> the rotated rows, fp64."""
    y = x.clone()
    pairs = cos_sin.shape[1] // 2
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for t in range(x.shape[0]):
        for i in range(pairs):
            p = positions[axis[i]][t]
            c, s = cos_sin[p, i].item(), cos_sin[p, pairs + i].item()
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def sees(j, context, mask, window, sinks):
    """Whether a drafted token with that mask sees position j."""
    if j >= context:
        return bool(mask >> (j - context) & 1)
    here = context + bin(mask).count("1") - 1
    return not window or j < sinks or j > here - window


def tree(q, k, v, table, lens, drafted, masks, page_size, scale, window=0, sinks=0):
    """q [B, T, Hq, d], caches [P, H, page_size, d] fp64, masks [B][T] of non-negative ints
    -> o, lse and the sums of the weighted magnitudes of v."""
    B, T, Hq, d = q.shape
    H = k.shape[1]
    G = Hq // H
    o, a = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, T, Hq), -math.inf, dtype=q.dtype)
    for b in range(B):
        context = lens[b] - drafted[b]
        for t in range(drafted[b]):
            mask = masks[b][t] & ((1 << drafted[b]) - 1)
            at = [j for j in range(lens[b]) if sees(j, context, mask, window, sinks)]
            if not at:
                continue
            pages = torch.tensor([int(table[b][j // page_size]) for j in at])
            place = torch.tensor([j % page_size for j in at])
            for h in range(H):
                r = slice(h * G, (h + 1) * G)
                o[b, t, r], lse[b, t, r], a[b, t, r] = ref.attend(
                    q[b, t, r], k[pages, h, place], v[pages, h, place], scale)
    return o, lse, a


def window(q, k, v, table, lens, page_size, scale, window, sinks):
    """One token per sequence: the drafted token of a tree of one."""
    o, lse, a = tree(q[:, None], k, v, table, lens, [1 if n else 0 for n in lens],
                     [[1]] * len(lens), page_size, scale, window, sinks)
    return o[:, 0], lse[:, 0], a[:, 0]


def keep(values, table, context, path, counts, page_size):
    """values [P, H, page_size, ...]: the rows of the paths moved, in place."""
    for b, n in enumerate(counts):
        rows = []
        for i in range(n):
            j = context[b] + path[b][i]
            rows.append(values[int(table[b][j // page_size]), :, j % page_size].clone())
        for i, r in enumerate(rows):
            j = context[b] + i
            values[int(table[b][j // page_size]), :, j % page_size] = r
    return values
