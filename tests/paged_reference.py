"""Plain implementations, in 64 bits on the CPU, of the operators over a paged
key-value cache: loops over sequences, heads and rows, straight from the
definitions.  Caches are given as the fp64 values that they hold."""
from __future__ import annotations

import math

import numpy as np
import torch


def round_e4m3(x):
    """Nearest multiple of each value's e4m3 step (3 mantissa bits, least step 2^-9), ties to
    the even multiple; |x| <= 448."""
    out = np.zeros_like(x)
    for i, a in np.ndenumerate(x):
        if a:
            step = 2.0 ** max(math.floor(math.log2(abs(a))) - 3, -9)
            out[i] = round(a / step) * step  # (python rounds ties to even)
    return out


def quantise_row(x):
    """A row (fp64) -> (its values once stored, its scale byte)."""
    if not np.isfinite(x).all():
        return np.full_like(x, math.nan), 255
    top = float(np.abs(x).max())
    if top == 0:
        return np.zeros_like(x), 127
    s = -126
    while top / 2.0 ** s > 448:
        s += 1
    return round_e4m3(x / 2.0 ** s) * 2.0 ** s, s + 127


def quantise_rows(x):
    """quantise_row of many finite rows at once ([..., d] fp64): the type's own rounding of the
    scaled rows."""
    top = x.abs().amax(-1, keepdim=True)
    s = torch.full_like(top, -126.0)
    for e in range(-126, 121):
        s = torch.where(top > 448 * 2.0 ** e, torch.full_like(s, e + 1.0), s)
    s = torch.where(top == 0, torch.zeros_like(s), s)
    return (x * 2.0 ** -s).float().to(torch.float8_e4m3fn).double() * 2.0 ** s


def gather(values, pages, n, page_size):
    """Positions 0..n-1 of one sequence: values [P, H, page_size, d] -> [H, n, d]."""
    if n == 0:
        return values[:0].new_zeros((values.shape[1], 0, values.shape[3]))
    parts = [values[int(pages[j // page_size]), :, j % page_size] for j in range(n)]
    return torch.stack(parts, 1)


def attend(q, k, v, scale):
    """q [G, d], k, v [n, d] -> (o, lse, sum of the weighted magnitudes of v), fp64."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=q.dtype), \
            torch.zeros_like(q)
    s = (q @ k.T) * scale
    p = torch.softmax(s, -1)
    return p @ v, torch.logsumexp(s, -1), p @ v.abs()


def decode(q, k, v, table, lens, page_size, scale):
    """q [B, Hq, d], caches [P, H, page_size, d], fp64 -> o, lse and the magnitudes of attend."""
    B, Hq, d = q.shape
    H = k.shape[1]
    G = Hq // H
    o, a = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros((B, Hq), dtype=q.dtype)
    for b in range(B):
        kk, vv = gather(k, table[b], lens[b], page_size), gather(v, table[b], lens[b], page_size)
        for h in range(H):
            r = slice(h * G, (h + 1) * G)
            o[b, r], lse[b, r], a[b, r] = attend(q[b, r], kk[h], vv[h], scale)
    return o, lse, a


def bounds_of(k, table, lens, page_size, new_tokens, bounds):
    """bounds [P, H, 2, d] (fp64, changed in place): the blocks with any of the newest positions."""
    for b, n in enumerate(lens):
        for i in range(max(0, n - new_tokens) // page_size, -(-n // page_size)):
            rows = k[int(table[b][i]), :, :min(page_size, n - i * page_size)]
            bounds[int(table[b][i]), :, 0] = rows.amin(1)
            bounds[int(table[b][i]), :, 1] = rows.amax(1)
    return bounds


def scores_of(q, bounds, table, lens, page_size):
    """-> scores [B, H, width] and the sums of their terms' magnitudes, fp64."""
    B, Hq, d = q.shape
    H, width = bounds.shape[1], table.shape[1]
    G = Hq // H
    s = torch.full((B, H, width), -math.inf, dtype=q.dtype)
    a = torch.zeros((B, H, width), dtype=q.dtype)
    for b, n in enumerate(lens):
        for i in range(-(-n // page_size)):
            lo, hi = bounds[int(table[b][i]), :, 0], bounds[int(table[b][i]), :, 1]
            for h in range(H):
                x = q[b, h * G:(h + 1) * G]
                terms = x.clamp(min=0) * hi[h] + x.clamp(max=0) * lo[h]
                s[b, h, i] = terms.sum(-1).max()
                a[b, h, i] = (x.abs() * torch.maximum(lo[h].abs(), hi[h].abs())).sum(-1).max()
    return s, a


def choose(scores, n, page_size, num_blocks, first, last):
    """One (sequence, head): the chosen block indexes, rising."""
    blocks = -(-n // page_size)

    def key(i):
        if i >= blocks - last:
            return (0, 0.0, i)
        if i < first:
            return (1, 0.0, i)
        return (2, 0.0, i) if math.isnan(scores[i]) else (3, -scores[i], i)

    return sorted(sorted(range(blocks), key=key)[:num_blocks])


def sparse(q, k, v, table, lens, page_size, scores, num_blocks, scale, first=0, last=1):
    B, Hq, d = q.shape
    H = k.shape[1]
    G = Hq // H
    o, a = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros((B, Hq), dtype=q.dtype)
    blocks = torch.full((B, H, num_blocks), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        kk, vv = gather(k, table[b], n, page_size), gather(v, table[b], n, page_size)
        for h in range(H):
            best = choose(scores[b, h].tolist(), n, page_size, num_blocks, first, last)
            blocks[b, h, :len(best)] = torch.tensor(best, dtype=torch.int32)
            keep = [j for i in best for j in range(i * page_size, min(n, (i + 1) * page_size))]
            r = slice(h * G, (h + 1) * G)
            o[b, r], lse[b, r], a[b, r] = attend(q[b, r], kk[h, keep], vv[h, keep], scale)
    return o, lse, a, blocks
