"""Single-token attention where magnitudes lie far apart: rows of zeros in a quantised cache,
weights far below the largest, queries of a wide range.  All against the plain 64-bit
implementation, over the values that the cache holds."""
import math

import numpy as np
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import TYPES, Cache, check_attention, make_table, pages_for, ref

pytestmark = pytest.mark.gpu


def filled(lens, heads, page_size, d, kind, k, v, seed=0):
    """A cache into which kv_cache_write has stored k, v [tokens, heads, d], sequence by sequence."""
    pages = pages_for(lens, page_size)
    cache = Cache(pages, heads, page_size, d, kind, seed=seed)
    table = make_table(lens, page_size, pages, seed=seed)
    slots = torch.cat([table[b, torch.arange(n) // page_size].long() * page_size
                       + torch.arange(n) % page_size for b, n in enumerate(lens)])
    fat.kv_cache_write(k.cuda(), v.cuda(), cache.k, cache.v, slots.cuda(), **cache.scale_args)
    return cache, table


def check(cache, table, lens, q, what=""):
    """Decode, whole and split as the lengths have it, against the 64-bit result."""
    o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda(),
                                   **cache.scale_args)
    assert fat.check_device_error() == fat.FAT_OK
    k, v = cache.held()
    want = ref.decode(q.double(), k, v, table, lens, cache.page_size,
                      float(np.float32(q.shape[-1] ** -0.5)))
    check_attention(o, lse, *want, what=what, kind=cache.kind)
    return o, lse


def sink_inputs(lens, heads, group, d, typ, gap, seed):
    """Queries near one direction of signs for each head, keys whose scores are near 0 but for the
    positions `at` of each sequence, which are `gap` above; values around a mean that is not 0."""
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    u = torch.sign(torch.randn((heads, d), generator=g))
    q = u[:, None] + 0.2 * torch.randn((len(lens), heads, group, d), generator=g)
    k = 0.2 * torch.randn((n, heads, d), generator=g)
    v = 0.3 + 0.2 * torch.randn((n, heads, d), generator=g)
    at, start = [], 0
    for m in lens:
        at += [start + m // 3, start + m - 1] if m > 1 else []
        start += m
    k[at] = u * (gap / math.sqrt(d))  # scale = 1 / sqrt(d): u . k / sqrt(d) = gap
    return (q.reshape(len(lens), heads * group, d).to(TYPES[typ]), k.to(TYPES[typ]), v, at)


@pytest.mark.parametrize("d,group", [(128, 4), (64, 1), (128, 16)])
@pytest.mark.parametrize("lens", [[200, 17], [8192, 700]], ids=["direct", "split"])
@pytest.mark.parametrize("typ,size,gap", [("bf16", 2.0 ** -9, 10.0), ("bf16", 2.0 ** -3, 12.0),
                                          ("fp16", 2.0 ** -3, 12.0)])
def test_e4m3_rows_of_zeros_with_the_highest_score(cuda_device, d, group, lens, typ, size, gap):
    """A row of zeros in V (a padding or null token) takes part in the softmax and adds nothing,
    whatever its scale; the other rows' weights keep their bits.

    The sums of magnitudes behind a score stay below 12 * 1.3, for which check_attention's 2^-12
    holds: 128 * 2^-24 * 15.6 = 1.2e-4, of the weight and of the total."""
    q, k, v, at = sink_inputs(lens, 2, group, d, typ, gap, seed=d + group)
    v = (v * size).to(TYPES[typ])
    v[at] = 0
    v[at[0]] = -0.0
    cache, table = filled(lens, 2, 32, d, "e4m3", k, v, seed=3)
    assert (cache.scales[1] == 127).any()
    check(cache, table, lens, q)
    # a row of zeros with any other scale byte, as another writer may leave it
    page, place = int(table[0, at[0] // 32]), at[0] % 32
    for byte in (1, 200, 254):
        cache.scales[1][page, :, place] = byte
        check(cache, table, lens, q, f"byte {byte}")
    # but 255 marks a row that reads as NaN
    cache.scales[1][page, :, place] = 255
    o, _ = check(cache, table, lens, q)
    assert torch.isnan(o[0]).all() and not torch.isnan(o[1]).any()


@pytest.mark.parametrize("typ", ["bf16", "fp16"])
@pytest.mark.parametrize("lens", [[100, 1], [3000, 900]], ids=["direct", "split"])
def test_e4m3_values_all_zeros(cuda_device, typ, lens):
    """V of nothing but zeros, with scores of +-300 so that 2^(r' - r) has no value to start from."""
    for sign in (1.0, -1.0):
        q, k, _, _ = sink_inputs(lens, 2, 4, 64, typ, 8.0, seed=5)
        u = torch.sign(q.float()).view(len(lens), 2, 4, 64)[0, :, 0]
        k = (sign * u * 37.5).expand(sum(lens), 2, 64).to(TYPES[typ])
        cache, table = filled(lens, 2, 16, 64, "e4m3", k, torch.zeros_like(k), seed=4)
        o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(),
                                       **cache.scale_args)
        assert torch.equal(o.cpu(), torch.zeros_like(q))
        want = ref.decode(q.double(), *cache.held(), table, lens, 16, 0.125)[1]
        assert want.abs().min() > 100
        # a score is off by at most 64 * 2^-24 of its sum of magnitudes, |want| here
        off = (lse.cpu().double() - want).abs() - 2.0 ** -18 * want.abs()
        assert off.max() <= 2.0 ** -21 * want.abs().max()


@pytest.mark.parametrize("typ,binades", [("bf16", 16), ("bf16", 23), ("bf16", 30), ("fp16", 16),
                                         ("fp16", 22)])
@pytest.mark.parametrize("d,group", [(128, 4), (64, 1), (64, 12)])
def test_e4m3_queries_of_a_wide_range(cuda_device, typ, binades, d, group):
    """Half of a query's elements lie `binades` below the others and decide alone: the keys are
    zero where the query is large.  The scores' standard deviation is 2, and their sums of
    magnitudes are below 15, for which check_attention's 2^-12 holds: 128 * 2^-24 * 15 = 1.14e-4,
    of the weight and of the total."""
    lens, heads = [300, 77], 2
    g = torch.Generator().manual_seed(binades + d)
    q = torch.randn((len(lens), heads * group, d), generator=g) * 2.0 ** 12
    q[..., d // 2:] *= 2.0 ** -binades
    k = torch.randn((sum(lens), heads, d), generator=g)
    k *= 2.0 * math.sqrt(2.0) * 2.0 ** (binades - 12)  # (sqrt(d / 2) terms, scale 1 / sqrt(d))
    k[..., :d // 2] = 0
    v = torch.randn((sum(lens), heads, d), generator=g)
    q, k, v = (t.to(TYPES[typ]) for t in (q, k, v))
    assert all(torch.isfinite(t).all() for t in (q, k, v))
    cache, table = filled(lens, heads, 16, d, "e4m3", k, v, seed=6)
    check(cache, table, lens, q)


def test_e4m3_queries_of_extreme_magnitude(cuda_device):
    """bf16 queries near the type's largest and least values, over keys that undo it."""
    lens, d = [100] * 6, 64
    g = torch.Generator().manual_seed(8)
    q = torch.randn((6, 1, d), generator=g)
    k = torch.randn((600, 1, d), generator=g)
    powers = [125, 110, 0, -110, -115, -124]
    for b, p in enumerate(powers):
        q[b] *= 2.0 ** p
        k[100 * b:100 * (b + 1)] *= 2.0 ** max(-110, min(110, -p))
        q[b] = q[b].clamp(-3e38, 3e38)
    v = torch.randn((600, 1, d), generator=g)
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    assert torch.isfinite(q).all() and (q != 0).float().mean() > 0.9
    cache, table = filled(lens, 1, 16, d, "e4m3", k, v, seed=7)
    o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda(),
                                   **cache.scale_args)
    kk, vv = cache.held()
    want = ref.decode(q.double(), kk, vv, table, lens, 16, 0.125)
    for b in (1, 2, 3):
        check_attention(o[b], lse[b], *(x[b] for x in want), what=f"2^{powers[b]}", kind="e4m3")
    # scores that a power more or less on one side makes huge (NaN only where fp32 has no value)
    # or nothing at all
    assert (lse[4:].cpu().double() - want[1][4:]).abs().max() <= 2e-4
    assert torch.isfinite(o[4:]).all()
