"""Single-token attention over the paged cache, whole and over chosen blocks,
and the block bounds and scores, against the plain 64-bit implementation."""
import math

import numpy as np
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import (BEHIND, TYPES, Cache, check_attention, make_table, pages_for, queries,
                           ref)

pytestmark = pytest.mark.gpu


def setup(lens, heads, group, page_size, d, q_type, kind, layout="phtd", seed=0, spread=0,
          width=None):
    pages = pages_for(lens, page_size)
    cache = Cache(pages, heads, page_size, d, kind, layout, seed=seed, spread=spread)
    if width is None:
        width = max(1, max(-(-n // page_size) for n in lens)) + 2
    table = make_table(lens, page_size, pages, seed=seed, width=width)
    q = queries(len(lens), heads * group, d, q_type, seed=seed)
    return cache, table, torch.tensor(lens, dtype=torch.int32), q


def run_decode(cache, table, lens, q, **kw):
    o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(), lens.cuda(),
                                   **cache.scale_args, **kw)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    return o, lse


def check_decode(cache, table, lens, q, what=""):
    scale = float(np.float32(q.shape[-1] ** -0.5))
    o, lse = run_decode(cache, table, lens, q)
    want = ref.decode(q.double(), cache.k_values, cache.v_values, table, lens.tolist(),
                      cache.page_size, scale)
    check_attention(o, lse, *want, what=what, kind=cache.kind)
    return o, lse


CASES = [
    # lens, heads, group, page_size, d, query type, cache type, layout
    ([1], 1, 1, 16, 128, "bf16", "bf16", "phtd"),
    ([0, 1, 2, 15, 16, 17], 2, 1, 16, 128, "bf16", "bf16", "phtd"),
    ([63, 64, 65, 0, 129, 200], 3, 4, 16, 128, "bf16", "bf16", "pthd"),
    ([300, 7, 511, 512, 513], 2, 8, 64, 128, "bf16", "e4m3", "phtd"),
    ([300, 7, 511, 0, 513], 2, 3, 16, 64, "fp16", "e4m3", "kv"),
    ([1000, 33], 1, 16, 32, 64, "fp16", "fp16", "kv"),
    ([100, 900], 2, 12, 128, 128, "fp16", "fp16", "phtd"),
    ([1500], 1, 33, 256, 128, "bf16", "bf16", "phtd"),
    ([700, 1], 1, 64, 16, 64, "bf16", "e4m3", "pthd"),
    ([1025, 40], 2, 5, 1024, 64, "bf16", "bf16", "phtd"),
    ([5000], 1, 2, 64, 64, "bf16", "e4m3", "phtd"),
    ([9001, 3], 1, 1, 16, 128, "bf16", "bf16", "phtd"),
    ([20] * 70, 1, 2, 16, 64, "bf16", "bf16", "phtd"),
    ([5] * 700 + [100], 1, 1, 16, 64, "bf16", "e4m3", "phtd"),
    ([0, 0, 0], 2, 2, 16, 128, "bf16", "bf16", "phtd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
def test_decode(cuda_device, case):
    lens, *rest = case
    cache, table, lens_t, q = setup(lens, *rest, seed=len(lens) + max(lens))
    check_decode(cache, table, lens_t, q, str(case))


def test_decode_one_sequence_across_all_blocks(cuda_device):
    """One sequence long enough that every thread block gets part of it, and more of them."""
    for lens in ([60000], [30000, 1, 25000, 0, 700]):
        cache, table, lens_t, q = setup(lens, 1, 2, 64, 64, "bf16", "e4m3", seed=3)
        scale = float(np.float32(64 ** -0.5))
        o, lse = run_decode(cache, table, lens_t, q)
        for b, n in enumerate(lens):  # (the pages at once: the loop of the reference is slow here)
            ids = table[b, :-(-n // 64)].long()
            k, v = (x[ids, 0].reshape(-1, 64)[:n] for x in (cache.k_values, cache.v_values))
            want = ref.attend(q[b].double(), k, v, scale)
            check_attention(o[b], lse[b], *want, what=f"{lens} {b}", kind="e4m3")


def test_decode_strided_queries_outputs_and_scale(cuda_device):
    lens = [40, 300]
    cache, table, lens_t, q = setup(lens, 2, 2, 16, 128, "bf16", "bf16", seed=8)
    wide = torch.zeros((2, 4 + 3, 128), dtype=torch.bfloat16)
    wide[:, 2:6] = q
    wide = wide.cuda()
    big = torch.full((4, table.shape[1] + 5), BEHIND, dtype=torch.int32)
    big[::2, :table.shape[1]] = table
    big = big.cuda()
    out = (torch.full((2, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((2, 4), 7.0, device="cuda"))
    work = torch.empty(fat.attn_decode_workspace_bytes(2, 4, 2, 128), dtype=torch.uint8,
                       device="cuda")
    work.fill_(255)  # any contents
    o, lse = fat.attn_decode_paged(wide[:, 2:6], cache.k, cache.v, big[::2, :table.shape[1]],
                                   lens_t.cuda(), 0.25, workspace=work, out=out)
    assert o is out[0] and lse is out[1]
    want = ref.decode(q.double(), cache.k_values, cache.v_values, table, lens, 16, 0.25)
    # scale 0.25 is 2.8 / sqrt(128): scores and their error grow by 2.8
    off = (o.cpu().double() - want[0]).abs()
    assert (off <= 2.0 ** -8 * want[0].abs() + 2.0 ** -10 * want[2]).all()
    assert ((lse.cpu().double() - want[1]).abs() <= 3e-4).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_what_lies_behind_a_sequence_has_no_part(cuda_device, kind):
    """NaN, infinities and huge values in the last page's free rows and in free pages."""
    lens = [1, 17, 31, 40, 0, 64, 100]
    cache, table, lens_t, q = setup(lens, 2, 4, 16, 128, "bf16", kind, seed=4)
    want_o, want_lse = check_decode(cache, table, lens_t, q)
    used = torch.zeros(cache.k.shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // 16], j % 16] = True
    free = ~used[:, None, :, None].cuda().expand(cache.k.shape)
    for fill in (math.nan, math.inf, -math.inf):
        for t in (cache.k, cache.v):
            raw = t.view(torch.uint8) if kind == "e4m3" else t
            # an e4m3 code has no infinity: its NaN code, and scale bytes of all kinds
            raw[free] = 0x7F if kind == "e4m3" else fill
        if kind == "e4m3":
            for s in cache.scales:
                s[~used[:, None, :].cuda().expand(s.shape)] = 255 if math.isnan(fill) else 254
        o, lse = run_decode(cache, table, lens_t, q)
        assert torch.equal(o, want_o) and torch.equal(lse, want_lse)


def test_nan_and_infinities_in_use(cuda_device):
    """A NaN key makes its sequence's heads NaN and no other's; so does an infinite logit; a NaN
    value makes its column NaN."""
    lens = [40, 40, 40, 40]
    cache, table, lens_t, q = setup(lens, 2, 2, 16, 64, "bf16", "bf16", seed=6)
    page = [int(table[b, 1]) for b in range(4)]
    for t, values, b, h, place, c, x in (
            (cache.k, cache.k_values, 0, 1, 3, 5, math.nan),
            (cache.v, cache.v_values, 2, 0, 9, 17, math.nan),
            (cache.v, cache.v_values, 3, 1, 2, 1, math.inf)):
        t[page[b], h, place, c] = x
        values[page[b], h, place, c] = x
    check_decode(cache, table, lens_t, q)


def test_e4m3_row_of_nan(cuda_device):
    cache, table, lens_t, q = setup([40, 70], 1, 4, 16, 128, "bf16", "e4m3", seed=9)
    cache.scales[0][table[0, 1].item(), 0, 3] = 255
    cache.k_values[table[0, 1].item(), 0, 3] = math.nan
    cache.scales[1][table[1, 2].item(), 0, 3] = 255
    cache.v_values[table[1, 2].item(), 0, 3] = math.nan
    check_decode(cache, table, lens_t, q)


@pytest.mark.parametrize("kind,q_type", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"),
                                         ("e4m3", "fp16")])
def test_values_of_unlike_magnitude(cuda_device, kind, q_type):
    """V rows whose magnitudes are up to 2^16 (fp16: 2^6) apart, with and without weight on the
    large ones: what rounds is relative to the weighted sum, not to the largest row."""
    lens = [200, 333]
    cache, table, lens_t, q = setup(lens, 1, 4, 16, 128, q_type, kind, seed=12,
                                    spread=3 if q_type == "fp16" else 8)
    g = torch.Generator().manual_seed(3)
    # plain keys again, but the rows with large values get no weight for half of the queries
    for b, n in enumerate(lens):
        big = torch.rand(n, generator=g) < 0.2
        for j in range(n):
            page, place = int(table[b, j // 16]), j % 16
            row = torch.randn(128, generator=g).double() * 0.5
            if big[j]:
                row = -6.0 * torch.sign(q[b, 0].double()) * row.abs()
            if kind == "e4m3":
                stored, e = ref.quantise_row(row.numpy())
                stored = torch.tensor(stored)
                cache.scales[0][page, 0, place] = e
                cache.k[page, 0, place] = (stored * 2.0 ** (127.0 - e)).float().to(
                    torch.float8_e4m3fn).cuda()
            else:
                stored = row.to(TYPES[kind]).double()
                cache.k[page, 0, place] = stored.to(TYPES[kind]).cuda()
            cache.k_values[page, 0, place] = stored
    # scores reach 6 * 0.08 * 128 * 0.64 * 0.09 ~ 4 times those of the other tests, and so does
    # their error: 2^-10 of the magnitudes, 4e-4 on the LSE; and the weights' own rounding
    weights = 2.0 ** -11 if kind == "e4m3" and q_type == "bf16" else 0.0
    o, lse = run_decode(cache, table, lens_t, q)
    want = ref.decode(q.double(), cache.k_values, cache.v_values, table, lens, 16,
                      float(np.float32(128 ** -0.5)))
    half = 2.0 ** -8 if q_type == "bf16" else 2.0 ** -11
    off = (o.cpu().double() - want[0]).abs()
    allowed = half * want[0].abs() + (2.0 ** -10 + weights) * want[2] + 2.0 ** -25
    assert (off <= allowed).all(), (off / allowed).max()
    assert ((lse.cpu().double() - want[1]).abs() <= 4e-4 + 2.0 ** -21 * want[1].abs()).all()


def test_large_logits(cuda_device):
    """Logits of several hundred: the running maximum grows by many binades, in both orders."""
    lens = [500, 500]
    cache, table, lens_t, q = setup(lens, 1, 3, 16, 64, "bf16", "bf16", seed=15)
    for b in range(2):
        for j in range(500):
            page, place = int(table[b, j // 16]), j % 16
            size = (j if b == 0 else 499 - j) / 8.0
            row = (torch.sign(q[b, 1].double()) * size / 8).to(torch.bfloat16)
            cache.k[page, 0, place] = row.cuda()
            cache.k_values[page, 0, place] = row.double()
    o, lse = run_decode(cache, table, lens_t, q)
    want = ref.decode(q.double(), cache.k_values, cache.v_values, table, lens, 16,
                      float(np.float32(64 ** -0.5)))
    # |logit| up to 8 * 64 * 0.8 / 8 = 51 natural units per unit scale ... the sum of magnitudes
    # is at most 7.8 * sum |q| * scale < 7.8 * 60 / 8 = 59: 64 * 2^-24 * 59 = 2.2e-4 a score
    off = (o.cpu().double() - want[0]).abs()
    assert (off <= 2.0 ** -8 * want[0].abs() + 2.0 ** -11 * want[2]).all()
    assert ((lse.cpu().double() - want[1]).abs() <= 3e-4 + 2.0 ** -21 * want[1].abs()).all()


def test_decode_is_the_same_every_time(cuda_device):
    cache, table, lens_t, q = setup([9000, 10, 3000], 2, 4, 64, 128, "bf16", "bf16", seed=16)
    first = run_decode(cache, table, lens_t, q)
    for _ in range(5):
        again = run_decode(cache, table, lens_t, q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_reports_a_bad_page_or_length(cuda_device):
    cache, table, lens_t, q = setup([40, 40], 1, 2, 16, 64, "bf16", "e4m3", seed=17)
    want = run_decode(cache, table, lens_t, q)
    bad = table.clone()
    for value in (-1, cache.k.shape[0], BEHIND, -2 ** 31):
        bad[0, 1] = value
        o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, bad.cuda(), lens_t.cuda(),
                                       **cache.scale_args)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX
        assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])
    for value in (-1, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        full = table.clone()
        full[full == BEHIND] = 0
        o, lse = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, full.cuda(),
                                       torch.tensor([value, 40], dtype=torch.int32).cuda(),
                                       **cache.scale_args)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX
        assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])


# ------------------------------------------------------------------ bounds and scores
@pytest.mark.parametrize("kind,q_type,d,page_size,group,new", [
    ("bf16", "bf16", 128, 16, 1, None), ("bf16", "bf16", 64, 64, 5, 1),
    ("fp16", "fp16", 128, 32, 8, 33), ("e4m3", "bf16", 128, 16, 16, 2),
    ("e4m3", "fp16", 64, 256, 3, None), ("bf16", "bf16", 128, 16, 20, 1)])
def test_bounds_and_scores(cuda_device, kind, q_type, d, page_size, group, new):
    lens = [1, 0, 15, 16, 17, 300, 555]
    cache, table, lens_t, q = setup(lens, 2, group, page_size, d, q_type, kind, "pthd", seed=d)
    typ = TYPES[q_type]
    bounds = torch.full((cache.k.shape[0], 2, 2, d), 99.0, dtype=typ, device="cuda")
    got = fat.kv_block_bounds(cache.k, table.cuda(), lens_t.cuda(), bounds, new,
                              k_scale=cache.scales[0])
    assert got is bounds
    want = ref.bounds_of(cache.k_values, table, lens, page_size, new or 10 ** 9,
                         torch.full(bounds.shape, 99.0, dtype=torch.float64))
    assert torch.equal(bounds.cpu().double(), want.to(typ).double())
    if new is not None:
        fat.kv_block_bounds(cache.k, table.cuda(), lens_t.cuda(), bounds,
                            k_scale=cache.scales[0])
    scores = fat.kv_block_scores(q.cuda(), bounds, table.cuda(), lens_t.cuda(), page_size)
    want, magnitude = ref.scores_of(q.double(), bounds.cpu().double(), table, lens, page_size)
    scores = scores.cpu().double()
    assert torch.equal(torch.isinf(scores), torch.isinf(want))
    fine = torch.isfinite(want)
    # 2 d products in fp32
    off = (scores - want).abs()[fine] / (2 * d * 2.0 ** -24 * magnitude[fine] + 1e-30)
    assert off.max() <= 1.0
    assert fat.check_device_error() == fat.FAT_OK
    # the scores do bound every key
    for b, n in enumerate(lens):
        k = ref.gather(cache.k_values, table[b], n, page_size)
        for h in range(2):
            x = q[b, h * group:(h + 1) * group].double()
            for j in range(n):
                top = (x @ k[h, j]).max()
                assert top <= want[b, h, j // page_size] + 1e-9


def test_bounds_and_scores_carry_nan(cuda_device):
    cache, table, lens_t, q = setup([40, 40], 1, 2, 16, 64, "bf16", "bf16", seed=2)
    cache.k[int(table[0, 1]), 0, 3, 7] = math.nan
    bounds = torch.zeros((cache.k.shape[0], 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    fat.kv_block_bounds(cache.k, table.cuda(), lens_t.cuda(), bounds)
    nan = torch.isnan(bounds)
    assert nan[int(table[0, 1]), 0, :, 7].all() and nan.sum() == 2
    scores = fat.kv_block_scores(q.cuda(), bounds, table.cuda(), lens_t.cuda(), 16)
    assert torch.isnan(scores).nonzero().tolist() == [[0, 0, 1]]


# ------------------------------------------------------------------ chosen blocks
def check_sparse(cache, table, lens_t, q, scores, num_blocks, first=0, last=1):
    o, lse, blocks = fat.attn_decode_sparse(
        q.cuda(), cache.k, cache.v, table.cuda(), lens_t.cuda(), scores.cuda(), num_blocks,
        first_blocks=first, last_blocks=last, **cache.scale_args)
    assert fat.check_device_error() == fat.FAT_OK
    *want, want_blocks = ref.sparse(q.double(), cache.k_values, cache.v_values, table,
                                    lens_t.tolist(), cache.page_size, scores.double(), num_blocks,
                                    float(np.float32(q.shape[-1] ** -0.5)), first, last)
    assert torch.equal(blocks.cpu(), want_blocks)
    check_attention(o, lse, *want, what=f"{num_blocks} {first} {last}",
                    kind=cache.kind)
    return o, lse, blocks


@pytest.mark.parametrize("kind,q_type,d,page_size,group", [
    ("bf16", "bf16", 128, 16, 4), ("e4m3", "bf16", 64, 32, 1), ("fp16", "fp16", 64, 16, 9),
    ("e4m3", "fp16", 128, 16, 16)])
@pytest.mark.parametrize("num_blocks,first,last", [(1, 0, 1), (3, 0, 0), (7, 2, 2), (500, 0, 1)])
def test_sparse(cuda_device, kind, q_type, d, page_size, group, num_blocks, first, last):
    lens = [0, 1, 16, 50, 401, 640]
    cache, table, lens_t, q = setup(lens, 2, group, page_size, d, q_type, kind, seed=21)
    g = torch.Generator().manual_seed(num_blocks)
    scores = torch.randn((len(lens), 2, table.shape[1]), generator=g)
    check_sparse(cache, table, lens_t, q, scores, num_blocks, first, last)


def test_sparse_ties_nan_and_infinities(cuda_device):
    """Equal scores take the lower index; -0 equals 0; NaN is above +inf; -inf can be chosen."""
    lens = [16 * 40 - 3] * 4
    cache, table, lens_t, q = setup(lens, 1, 1, 16, 64, "bf16", "bf16", seed=23)
    g = torch.Generator().manual_seed(1)
    scores = torch.randint(0, 3, (4, 1, table.shape[1]), generator=g).float()
    scores[1] = torch.where(torch.rand(table.shape[1], generator=g) < 0.5, 0.0, -0.0)
    scores[2] = -math.inf
    scores[2, 0, 7] = -5.0
    scores[3, 0, 5], scores[3, 0, 9], scores[3, 0, 2] = math.nan, math.inf, -math.nan
    scores[3, 0, 30] = -math.inf
    for num_blocks in (1, 2, 5, 17, 39, 40):
        for last in (0, 1):
            check_sparse(cache, table, lens_t, q, scores, num_blocks, 0, last)


def test_sparse_of_many_blocks(cuda_device):
    """More blocks than threads, scores that agree in their leading bits."""
    n, ps = 16 * 5000 - 7, 16
    cache, table, lens_t, q = setup([n], 1, 2, ps, 64, "bf16", "e4m3", seed=25)
    g = torch.Generator().manual_seed(4)
    width = table.shape[1]
    for kind in range(3):
        scores = {0: torch.randn(width, generator=g),
                  1: 1.0 + torch.randint(0, 300, (width,), generator=g) * 2.0 ** -22,
                  2: torch.zeros(width)}[kind].float().view(1, 1, width)
        for num_blocks in (1, 64, 1700, 4999):
            blocks = fat.attn_decode_sparse(q.cuda(), cache.k, cache.v, table.cuda(),
                                            lens_t.cuda(), scores.cuda(), num_blocks,
                                            **cache.scale_args)[2]
            want = ref.choose(scores[0, 0].tolist(), n, ps, num_blocks, 0, 1)
            assert blocks[0, 0].cpu().tolist() == want


@pytest.mark.parametrize("count", [8192, 8193, 32768, 33000])
def test_sparse_of_very_many_blocks(cuda_device, count):
    """A sequence whose table repeats a few pages, around the counts where the choice changes its
    way: the blocks, and the attention over the first and the last of them."""
    n, ps, d = 16 * count - 5, 16, 64
    cache = Cache(8, 1, ps, d, "bf16", seed=count)
    g = torch.Generator().manual_seed(count)
    table = torch.randint(0, 8, (1, count + 3), generator=g, dtype=torch.int32)
    q = queries(1, 2, d, "bf16", seed=count)
    scores = torch.randn((1, 1, count + 3), generator=g)
    scores[0, 0, ::7] = scores[0, 0, 3]  # many equal ones
    for num_blocks in (5, count // 3, count - 1, count + 1):
        o, lse, blocks = fat.attn_decode_sparse(
            q.cuda(), cache.k, cache.v, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
            scores.cuda(), num_blocks)
        want = ref.choose(scores[0, 0].tolist(), n, ps, num_blocks, 0, 1)
        got = blocks[0, 0].cpu().tolist()
        assert got[:len(want)] == want and set(got[len(want):]) <= {-1}
        keep = torch.tensor(want)
        place = (keep[:, None] * ps + torch.arange(ps)).flatten()
        ids = table[0].long()[keep]
        k, v = (x[ids, 0].reshape(-1, d)[place < n] for x in (cache.k_values, cache.v_values))
        check_attention(o, lse, *(x[None] for x in ref.attend(q[0].double(), k, v, 0.125)),
                        what=f"{count} {num_blocks}")
    assert fat.check_device_error() == fat.FAT_OK


def test_sparse_of_many_sequences(cuda_device):
    """More (sequence, head) pairs than threads in a block."""
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 70, (90,), generator=g).tolist()
    cache, table, lens_t, q = setup(lens, 3, 2, 16, 64, "fp16", "e4m3", seed=28)
    check_sparse(cache, table, lens_t, q, torch.randn((90, 3, table.shape[1]), generator=g), 2)


def test_all_blocks_chosen_equals_the_whole(cuda_device):
    lens = [100, 0, 640, 333]
    cache, table, lens_t, q = setup(lens, 2, 4, 16, 128, "bf16", "bf16", seed=27)
    scores = torch.randn((4, 2, table.shape[1]))
    want = check_decode(cache, table, lens_t, q)
    got = check_sparse(cache, table, lens_t, q, scores, 40)
    assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -6  # a step at magnitudes < 4


# ------------------------------------------------------------------ as used together
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_few_decoding_steps(cuda_device, kind):
    """Prompts are written, the prefix is read back for their attention, then a few steps append
    a token, renew the bounds, score, and attend (whole and sparse); the last one again from a
    captured graph, with lengths that change between its replays."""
    H, G, d, ps, steps = 2, 4, 128, 16, 5
    start = [5, 70, 31]
    lens = [n + steps for n in start]
    pages = pages_for(lens, ps)
    cache = Cache(pages, H, ps, d, kind, seed=31)
    table = make_table(lens, ps, pages, seed=31)
    dev_table = table.cuda()
    g = torch.Generator().manual_seed(33)
    typ = torch.bfloat16
    bounds = torch.zeros((pages, H, 2, d), dtype=typ, device="cuda")
    tokens = [torch.randn((n, 2, H, d), generator=g).to(typ) for n in lens]

    def slot(b, j):
        return int(table[b, j // ps]) * ps + j % ps

    slots = torch.tensor([slot(b, j) for b, n in enumerate(start) for j in range(n)])
    x = torch.cat([t[:n] for t, n in zip(tokens, start)]).cuda()
    fat.kv_cache_write(x[:, 0], x[:, 1], cache.k, cache.v, slots.cuda(), **cache.scale_args)
    now = torch.tensor(start, dtype=torch.int32, device="cuda")
    fat.kv_block_bounds(cache.k, dev_table, now, bounds, k_scale=cache.scales[0])
    # the second prompt's last 8 tokens attend to its prefix, read back as one tensor
    k, v = fat.kv_cache_read(cache.k, cache.v, dev_table[1:2], now[1:2], 70, dtype=typ,
                             **cache.scale_args)
    qs = torch.randn((1, H, 8, d), generator=g).to(typ)
    o, lse = fat.attn_fwd_splitkv(qs.cuda(), k, v, causal=True)
    held = cache.held()
    kk, vv = (ref.gather(t, table[1], 70, ps) for t in held)
    for i in range(8):
        for h in range(H):
            want = ref.attend(qs[0, h, i:i + 1].double(), kk[h, :63 + i], vv[h, :63 + i],
                              float(np.float32(d ** -0.5)))
            assert (o[0, h, i].cpu().double() - want[0][0]).abs().max() <= 2e-2
            assert abs(lse[0, h, i].item() - want[1].item()) <= 1e-3

    def step(q, k1, v1, slots1, lens1, num_blocks):
        fat.kv_cache_write(k1, v1, cache.k, cache.v, slots1, **cache.scale_args)
        fat.kv_block_bounds(cache.k, dev_table, lens1, bounds, 1, k_scale=cache.scales[0])
        scores = fat.kv_block_scores(q, bounds, dev_table, lens1, ps)
        whole = fat.attn_decode_paged(q, cache.k, cache.v, dev_table, lens1, **cache.scale_args)
        best = fat.attn_decode_sparse(q, cache.k, cache.v, dev_table, lens1, scores, num_blocks,
                                      **cache.scale_args)
        return whole, scores, best

    def check(q, lens1, result):
        whole, scores, best = result
        held = cache.held()
        scale = float(np.float32(d ** -0.5))
        check_attention(*whole, *ref.decode(q.cpu().double(), *held, table, lens1, ps, scale),
                        kind=kind)
        want, magnitude = ref.scores_of(
            q.cpu().double(), ref.bounds_of(held[0], table, lens1, ps, 10 ** 9,
                                            torch.zeros(bounds.shape, dtype=torch.float64)),
            table, lens1, ps)
        fine = torch.isfinite(want)
        assert ((scores.cpu().double() - want).abs()[fine]
                <= (2 * d * 2.0 ** -24 * magnitude)[fine] + 1e-30).all()
        *att, chosen = ref.sparse(q.cpu().double(), *held, table, lens1, ps,
                                  scores.cpu().double(), 3, scale)
        assert torch.equal(best[2].cpu(), chosen)
        check_attention(best[0], best[1], *att, kind=kind)

    inputs = []
    for i in range(steps):
        lens1 = [n + i + 1 for n in start]
        x = torch.stack([tokens[b][n - 1] for b, n in enumerate(lens1)]).cuda()
        inputs.append((queries(3, H * G, d, "bf16", seed=40 + i).cuda(), x[:, 0], x[:, 1],
                       torch.tensor([slot(b, n - 1) for b, n in enumerate(lens1)]).cuda(),
                       torch.tensor(lens1, dtype=torch.int32).cuda()))
    for i in range(3):
        check(inputs[i][0], inputs[i][4].tolist(), step(*inputs[i], 3))
    # the last steps as replays of one graph
    static = [t.clone() for t in inputs[3]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static, 3)  # (writes the same tokens as the first replay)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = step(*static, 3)
    for i in (3, 4):
        for a, b in zip(static, inputs[i]):
            a.copy_(b)
        graph.replay()
        check(static[0], static[4].tolist(), result)
    assert fat.check_device_error() == fat.FAT_OK


def test_calls_on_two_streams_at_once(cuda_device):
    """Each call has a workspace of its own: two streams give what one gives."""
    a = setup([4000, 100], 2, 4, 64, 128, "bf16", "bf16", seed=51)
    b = setup([3000, 2500, 9], 2, 4, 64, 128, "bf16", "e4m3", seed=52)
    dev = [(c, t.cuda(), n.cuda(), q.cuda()) for c, t, n, q in (a, b)]
    want = [fat.attn_decode_paged(q, c.k, c.v, t, n, **c.scale_args) for c, t, n, q in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, (c, t, n, q) in enumerate(dev):
            got[i].append(fat.attn_decode_paged(q, c.k, c.v, t, n, stream=streams[i],
                                                **c.scale_args))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[0], o) and torch.equal(w[1], l) for o, l in g)


def test_calls_from_several_threads(cuda_device):
    """Host threads with a stream each, writing to caches of their own and attending to them."""
    import threading

    made = [setup([1500 + 300 * i, 40, 900], 2, 4, 32, 128, "bf16", ("bf16", "e4m3")[i % 2],
                  seed=70 + i) for i in range(4)]
    dev = [(c, t.cuda(), n.cuda(), q.cuda()) for c, t, n, q in made]
    token = torch.randn((3, 2, 128), device="cuda").to(torch.bfloat16)

    def slots(i):  # the newest position of each sequence
        _, t, n, _ = made[i]
        return torch.tensor([int(t[b, (int(n[b]) - 1) // 32]) * 32 + (int(n[b]) - 1) % 32
                             for b in range(3)]).cuda()

    def run(i, out, times):
        c, t, n, q = dev[i]
        for _ in range(times):
            fat.kv_cache_write(token, token, c.k, c.v, at[i], **c.scale_args)
            out.append(fat.attn_decode_paged(q, c.k, c.v, t, n, **c.scale_args))

    at = [slots(i) for i in range(4)]
    want, got, errors = [[] for _ in dev], [[] for _ in dev], []
    for i in range(4):
        run(i, want[i], 1)
    torch.cuda.synchronize()

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                run(i, got[i], 12)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # told by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for w, g in zip(want, got):
        assert len(g) == 12
        assert all(torch.equal(w[0][0], o) and torch.equal(w[0][1], l) for o, l in g)
    assert fat.check_device_error() == fat.FAT_OK


def test_on_the_current_stream(cuda_device):
    """Calls go to torch's current stream, also where it is not the default one."""
    cache, table, lens_t, q = setup([3000, 77], 2, 4, 64, 128, "bf16", "e4m3", seed=53)
    want = run_decode(cache, table, lens_t, q)
    args = (torch.zeros_like(q.cuda()), cache.k, cache.v, table.cuda(), lens_t.cuda())
    real = q.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()) as _:
        torch.cuda._sleep(2_000_000)  # a call on another stream would see the zeros
        args[0].copy_(real)
        o, lse = fat.attn_decode_paged(*args, **cache.scale_args)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_graphs_share_a_workspace(cuda_device):
    """Two captured calls of different shapes with one workspace, replayed in turn."""
    work = torch.empty(fat.attn_decode_workspace_bytes(2, 8, 2, 128, 40), dtype=torch.uint8,
                       device="cuda")
    work.fill_(0xA5)
    graphs, want, got, keep = [], [], [], []  # (keep: a graph does not own its inputs)
    for i, lens in enumerate(([5000, 700], [1300, 4000])):
        cache, table, lens_t, q = setup(lens, 2, 4, 64, 128, "bf16", ("bf16", "e4m3")[i],
                                        seed=60 + i)
        scores = torch.randn((2, 2, table.shape[1]), generator=torch.Generator().manual_seed(i))
        args = (q.cuda(), cache.k, cache.v, table.cuda(), lens_t.cuda())
        scores = scores.cuda()

        def call(args=args, scores=scores, kw=cache.scale_args):
            whole = fat.attn_decode_paged(*args, workspace=work, **kw)
            return (*whole, *fat.attn_decode_sparse(*args, scores, 40, workspace=work, **kw))

        keep.append((args, scores, cache))
        want.append([t.clone() for t in call()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(call())
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1, 0, 0):
        for t in got[i]:
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_refusals(cuda_device):
    cache, table, lens, q = setup([40], 2, 2, 16, 64, "bf16", "bf16", width=40)
    table, lens, q = table.cuda(), lens.cuda(), q.cuda()
    good = dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=table, seq_lens=lens)
    for bad in (dict(q=q[:, :3]), dict(q=q.half()), dict(q=q.float()), dict(q=q.cpu()),
                dict(q=q[:, :, :32]), dict(page_table=table.long()), dict(seq_lens=lens.long()),
                dict(page_table=table[0]), dict(v_cache=cache.v[:, :1]),
                dict(out=(q.float(), torch.zeros((1, 4), device="cuda"))),
                dict(workspace=torch.zeros(10, device="cuda"))):
        with pytest.raises(ValueError):
            fat.attn_decode_paged(**{**good, **bad})
    for bad in (dict(scale=0.0), dict(scale=math.nan),
                dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fat.FatError, match="INVALID_ARG"):
            fat.attn_decode_paged(**{**good, **bad})
    scores = torch.zeros((1, 2, table.shape[1]), device="cuda")
    for bad in (dict(num_blocks=0), dict(num_blocks=2, first_blocks=2), dict(last_blocks=-1),
                dict(scores=scores[..., :1]), dict(scores=scores.half())):
        with pytest.raises(ValueError):
            fat.attn_decode_sparse(**{**good, "scores": scores, "num_blocks": 4, **bad})
    bounds = torch.zeros((cache.k.shape[0], 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(new_tokens=0), dict(bounds=bounds[:1]), dict(bounds=bounds.half())):
        with pytest.raises(ValueError):
            fat.kv_block_bounds(**{**dict(k_cache=cache.k, page_table=table, seq_lens=lens,
                                          bounds=bounds), **bad})
    with pytest.raises(ValueError):
        fat.kv_block_scores(q.half(), bounds, table, lens, 16)
    with pytest.raises(fat.FatError, match="INVALID_ARG"):
        fat.kv_block_scores(q, bounds, table, lens, 20)
