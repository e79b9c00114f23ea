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


@pytest.mark.parametrize("kind,typ", [("fp16", "fp16"), ("bf16", "bf16"), ("e4m3", "fp16"),
                                      ("e4m3", "bf16")])
@pytest.mark.parametrize("lens", [[200, 17], [8192, 700]], ids=["direct", "split"])
@pytest.mark.parametrize("gap", [14.0, 15.3, 16.1, 17.2, 18.5, 19.4, 20.3])
def test_weights_far_below_the_largest(cuda_device, kind, typ, lens, gap):
    """One key's score is `gap` above all others, which are equal (their weights round alike), and
    its value is zero in all columns but one: the others alone make up the rest.

    fp16 weights are off by at most 2^-25 where the largest is at least 2^11, of an e4m3 cache in
    units of p_j 2^s_j with s_j the power that scales row j: 2^-36 max_j (p_j 2^s_j) of the sum of
    the codes' magnitudes, v_j / 2^s_j, beside what check_attention allows."""
    d, group, heads = 64, 4, 1
    q, k, v, at = sink_inputs(lens, heads, group, d, typ, gap, seed=21)
    sink = k[at].clone()
    k.zero_()
    k[at] = sink
    v[at] = 0
    v[at, :, 7] = 1.0
    v = (v * (1.0 if kind == "bf16" else 64.0)).to(TYPES[typ])
    cache, table = filled(lens, heads, 16, d, kind, k, v, seed=9)
    o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda(),
                                   **cache.scale_args)
    kk, vv = cache.held()
    scale = float(np.float32(d ** -0.5))
    want = ref.decode(q.double(), kk, vv, table, lens, 16, scale)
    if kind != "bf16":
        power = torch.ones(vv.shape[:3], dtype=torch.float64) if kind == "fp16" \
            else 2.0 ** (cache.scales[1].cpu().double() - 127)
        for b, n in enumerate(lens):
            x = ref.gather(kk, table[b], n, 16)[0]
            s = ref.gather(power[..., None], table[b], n, 16)[0]
            codes = (ref.gather(vv, table[b], n, 16)[0] / s).abs().sum(0)
            for h in range(group):
                p = torch.softmax((x @ q[b, h].double()) * scale, 0)
                # (as part of the magnitudes, of which check_attention allows 2^-12)
                want[2][b, h] += 2.0 ** 12 * 2.0 ** -36 * (p[:, None] * s).max() * codes
    check_attention(o, lse, *want, kind=kind)


@pytest.mark.parametrize("typ", ["bf16", "fp16"])
@pytest.mark.parametrize("lens", [[300], [6000]], ids=["direct", "split"])
def test_infinite_values_of_little_weight(cuda_device, typ, lens):
    """An infinite value makes its column infinite, 20 nats (2^-29 of the largest weight) below the
    largest score as well."""
    d = 64
    q, k, v, at = sink_inputs(lens, 1, 4, d, typ, 1.0, seed=31)
    u = torch.sign(k[at[0], 0])
    k = k * 0.02
    k[at[0]] = u * (20.0 / math.sqrt(d))
    low = [5, 110, 111, 250, lens[0] - 2]
    for i, (j, gap) in enumerate(zip(low, (0.0, 4.0, 8.0, 12.0, 17.0))):
        k[j] = u * (gap / math.sqrt(d))
        v[j, 0, 2 * i] = math.inf
        v[j, 0, 2 * i + 1] = -math.inf
    cache, table = filled(lens, 1, 16, d, typ, k.to(TYPES[typ]), v.to(TYPES[typ]), seed=9)
    o, _ = check(cache, table, lens, q)
    assert torch.isinf(o[0, :, :10]).all() and torch.isfinite(o[0, :, 10:]).all()


@pytest.mark.parametrize("typ", ["bf16", "fp16"])
@pytest.mark.parametrize("lens", [[300, 40], [6000, 40]], ids=["direct", "split"])
def test_infinite_keys(cuda_device, typ, lens):
    """A score of +inf has no softmax: NaN, for the heads whose query is positive there; a score of
    -inf has no weight.  The other sequence is as it was."""
    d = 64
    q, k, v, _ = sink_inputs(lens, 1, 4, d, typ, 2.0, seed=32)
    q[0, :, 3] = torch.tensor([1.0, -1.0, 0.5, -0.25])
    k[77, 0, 3] = math.inf
    cache, table = filled(lens, 1, 16, d, typ, k.to(TYPES[typ]), v.to(TYPES[typ]), seed=9)
    o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda())
    want = ref.decode(q.double(), *cache.held(), table, lens, 16, 0.125)
    assert torch.isnan(want[0][0, ::2]).all() and torch.isfinite(want[0][0, 1::2]).all()
    assert torch.isnan(o[0, ::2]).all() and not torch.isfinite(lse[0, ::2]).any()
    check_attention(o[0, 1::2], lse[0, 1::2], *(x[0, 1::2] for x in want), kind=typ)
    check_attention(o[1], lse[1], *(x[1] for x in want), kind=typ)


@pytest.mark.parametrize("d,group", [(128, 4), (64, 1), (128, 16), (64, 16)])
def test_e4m3_weights_keep_more_bits_than_the_output(cuda_device, d, group):
    """Two values that nearly cancel under weights near 2/3 and 1/3: a rounding of the weights to
    11 bits would show in a bf16 output.  The scores' sums of magnitudes are below 1.5 (a key of
    signs times 0.7 / sqrt(d)), so a weight and the total are each off by less than
    128 * 2^-24 * 1.5 = 1.2e-5, together less than 2^-15, and the rest (2^-22 of an exponential,
    2^-16 of a weight in two parts) below that again: 2^-14 of the sum of p_j |v_j|."""
    heads, b = 2, 150
    g = torch.Generator().manual_seed(d + group)
    lens = [2] * b
    u = torch.sign(torch.randn((heads, d), generator=g))
    q = u[:, None] + 0.2 * torch.randn((b, heads, group, d), generator=g)
    q = q.reshape(b, heads * group, d).to(torch.bfloat16)
    k = torch.zeros((2 * b, heads, d))
    k[::2] = u * (0.66 / math.sqrt(d))
    v = torch.full((2 * b, heads, d), -1.0)
    v[::2] = 0.5
    cache, table = filled(lens, heads, 16, d, "e4m3", k.to(torch.bfloat16), v.to(torch.bfloat16),
                          seed=2)
    o, _ = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), **cache.scale_args)
    want = ref.decode(q.double(), *cache.held(), table, lens, 16, float(np.float32(d ** -0.5)))
    off = (o.cpu().double() - want[0]).abs()
    assert want[0].abs().min() < 1e-3  # (where the output's own rounding is far below the rest)
    assert (off <= 2.0 ** -8 * want[0].abs() + 2.0 ** -14 * want[2]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_infinite_queries(cuda_device, kind):
    """Scores of -inf alone leave nothing to weigh, as for an empty sequence, whatever finite
    elements stand beside the infinite one; +inf and NaN have no softmax."""
    g = torch.Generator().manual_seed(4)
    k = torch.randn((50, 1, 64), generator=g)
    k[:, 0, 0], k[:, 0, 1] = -1.0, 1.0
    q = torch.randn((1, 4, 64), generator=g)
    q[0, 0, :2] = torch.tensor([math.inf, 3e38])
    q[0, 1, 0] = -math.inf
    q[0, 2, 5] = math.nan
    v = torch.randn((50, 1, 64), generator=g)
    cache, table = filled([50], 1, 16, 64, kind, k.to(torch.bfloat16), v.to(torch.bfloat16))
    q = q.to(torch.bfloat16)
    o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(),
                                   torch.tensor([50], dtype=torch.int32).cuda(),
                                   **cache.scale_args)
    assert (o[0, 0] == 0).all() and lse[0, 0] == -math.inf
    assert torch.isnan(o[0, 1:3]).all() and not torch.isfinite(lse[0, 1:3]).any()
    want = ref.decode(q.double(), *cache.held(), table, [50], 16, 0.125)
    check_attention(o[0, 3], lse[0, 3], *(x[0, 3] for x in want), kind=kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_short_sequences_in_a_wide_table(cuda_device, kind):
    """A table as wide as a model's longest context, as a captured graph needs it: lengths from none
    to a few pages, then one that grew; entries behind a sequence are never used."""
    ps, H, G, d, width = 16, 2, 4, 128, 131072 // 16
    for lens in ([1, 0, 15, 16, 17, 200, 511], [513, 3, 0, 5000]):
        pages = pages_for(lens, ps)
        cache = Cache(pages, H, ps, d, kind, seed=len(lens))
        table = make_table(lens, ps, pages, seed=1, width=width)
        g = torch.Generator().manual_seed(len(lens))
        q = torch.randn((len(lens), H * G, d), generator=g).to(torch.bfloat16)
        check(cache, table, lens, q)
        args = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
        bounds = torch.zeros((pages, H, 2, d), dtype=torch.bfloat16, device="cuda")
        fat.kv_block_bounds(cache.k, *args, bounds, k_scale=cache.scales[0])
        scores = fat.kv_block_scores(q.cuda(), bounds, *args, ps).cpu()
        narrow = -(-max(lens) // ps)
        want, size = ref.scores_of(q.double(), bounds.cpu().double(), table[:, :narrow], lens, ps)
        assert (scores[..., narrow:] == -math.inf).all()
        got = scores[..., :narrow].double()
        fine = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), fine)
        # 2 d products in fp32
        assert ((got - want).abs()[fine] <= 2 * d * 2.0 ** -24 * size[fine]).all()
        o, lse, blocks = fat.attn_decode_sparse(q.cuda(), cache.k, cache.v, *args, scores.cuda(),
                                                9, **cache.scale_args)
        *att, chosen = ref.sparse(q.double(), *cache.held(), table, lens, ps, scores.double(), 9,
                                  float(np.float32(d ** -0.5)))
        assert torch.equal(blocks.cpu(), chosen)
        check_attention(o, lse, *att, kind=kind)
        assert fat.check_device_error() == fat.FAT_OK
