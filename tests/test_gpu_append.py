"""Storing tokens with their rotation against the plain 64-bit implementation, and bit by bit
against the same formula in fp32."""
import math

import pytest
import torch

import drafted_reference
import paged_reference as ref
import tensorized_online_softmax_gb300 as fat
from drafted_helpers import angle_table
from paged_helpers import HALF, TYPES, Cache

pytestmark = pytest.mark.gpu

CASES = [
    # tokens, q heads, heads, page size, d, type, cache type, layout, rotated, sections, interleaved
    (1, 1, 1, 16, 64, "bf16", "bf16", "phtd", 64, None, False),
    (5, 8, 2, 16, 128, "bf16", "bf16", "phtd", 128, None, False),
    (37, 6, 3, 32, 128, "fp16", "fp16", "pthd", 64, None, False),
    (37, 5, 5, 16, 64, "fp16", "fp16", "kv", 16, None, True),
    (40, 7, 1, 64, 128, "bf16", "e4m3", "kv", 128, (16, 24, 24), False),
    (40, 4, 2, 16, 128, "fp16", "e4m3", "phtd", 112, (0, 1, 50, 5), True),
    (33, 3, 3, 128, 64, "bf16", "e4m3", "pthd", 48, (24,), False),
    (300, 2, 1, 16, 64, "bf16", "bf16", "phtd", 32, (3, 13), True),
    (2100, 9, 3, 64, 128, "bf16", "e4m3", "phtd", 96, None, False),
    (2100, 13, 5, 64, 64, "fp16", "fp16", "phtd", 64, None, True),
]


def setup(tokens, Hq, H, page_size, d, typ, kind, layout, n, sections, seed=0, rows=500):
    g = torch.Generator().manual_seed(seed)
    pages = -(-tokens // page_size) + 3
    cache = Cache(pages, H, page_size, d, kind, layout, seed=seed)
    slots = torch.randperm(pages * page_size, generator=g)[:tokens]
    if tokens > 4:
        slots[2] = -1
    axes = len(sections) if sections else 1
    positions = torch.randint(0, rows, (axes, tokens), generator=g)
    positions[0, 0], positions[-1, -1] = 0, rows - 1
    x = [torch.randn((tokens, h, d), generator=g).to(TYPES[typ]) for h in (Hq, H, H)]
    return cache, slots, positions, angle_table(rows, n), x


def plain(x, table, positions, sections, interleaved):
    """The rotation in fp32, every product and sum rounded by itself."""
    pairs = table.shape[1] // 2
    axis = [a for a, n in enumerate(sections or (pairs,)) for _ in range(n)]
    i = torch.arange(pairs)
    at = positions[torch.tensor(axis)].T  # [T, pairs]
    c, s = table[at, i][:, None], table[at, pairs + i][:, None]
    y = x.float().clone()
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    a, b = x[..., lo].float(), x[..., hi].float()
    y[..., lo] = a * c - b * s
    y[..., hi] = b * c + a * s
    return y


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_append(cuda_device, case):
    tokens, Hq, H, page_size, d, typ, kind, layout, n, sections, interleaved = case
    cache, slots, positions, table, (q, k, v) = setup(*case[:-2], sections, seed=tokens)
    before = cache.held()
    given = positions if sections else positions[0]
    out = fat.kv_cache_append(q.cuda(), k.cuda(), v.cuda(), cache.k, cache.v, slots.cuda(),
                              given.cuda(), table.cuda(), sections=sections,
                              interleaved=interleaved, **cache.scale_args)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    args = table, positions, sections, interleaved
    assert torch.equal(out.cpu(), plain(q, *args).to(q.dtype))
    # the same rotation in 64 bits: two products and a sum of fp32, then the type's rounding
    few = slice(0, 40)
    want = drafted_reference.rotate(q[few].double(), table.double(), positions[:, few].tolist(),
                                    sections or (n // 2,), interleaved)
    slack = 2.0 ** -22 * q[few].double().abs().amax(-1, keepdim=True) + 2.0 ** -25
    assert ((out[few].cpu().double() - want).abs() <= HALF[q.dtype] * want.abs() + slack).all()
    for now, was, x in zip(cache.held(), before, (plain(k, *args), v.float())):
        rows = ref.quantise_rows(x.double()) if kind == "e4m3" else x.to(k.dtype).double()
        for t in range(tokens):
            if slots[t] >= 0:
                was[slots[t] // page_size, :, slots[t] % page_size] = rows[t]
        assert torch.equal(now, was)


def test_strided_inputs_in_place_and_without_queries(cuda_device):
    cache, slots, positions, table, _ = setup(20, 4, 2, 16, 128, "bf16", "bf16", "phtd", 128, None)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((20, 8, 128), generator=g).to(torch.bfloat16)  # one projection's output
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    args = table, positions, None, False
    dev = qkv.cuda()
    wide = torch.full((500, 160), 7.0)
    wide[:, :128] = table
    wide = wide.cuda()[:, :128]
    steps = torch.stack([positions[0], positions[0] + 1], 1).cuda()  # [20, 2]: every second entry
    out = torch.empty((20, 4, 128), dtype=torch.bfloat16, device="cuda")
    got = fat.kv_cache_append(dev[:, :4], dev[:, 4:6], dev[:, 6:], cache.k, cache.v, slots.cuda(),
                              steps[:, 0], wide, out=out)
    assert got is out and torch.equal(out.cpu(), plain(q, *args).bfloat16())
    first = [x.clone() for x in cache.held()]
    # in place
    mine = q.contiguous().cuda()
    got = fat.kv_cache_append(mine, dev[:, 4:6], dev[:, 6:], cache.k, cache.v, slots.cuda(),
                              positions[0].cuda(), table.cuda(), out=mine)
    assert got is mine and torch.equal(mine.cpu(), out.cpu())
    # keys and values only, and no token at all
    cache.k.zero_(), cache.v.zero_()
    assert fat.kv_cache_append(None, dev[:, 4:6], dev[:, 6:], cache.k, cache.v, slots.cuda(),
                               positions[0].cuda(), table.cuda()) is None
    for t in range(20):
        if slots[t] >= 0:
            at = slots[t] // 16, slice(None), slots[t] % 16
            assert all(torch.equal(a[at], b[at]) for a, b in zip(cache.held(), first))
    none = slots[:0].cuda()
    got = fat.kv_cache_append(dev[:0, :4], dev[:0, 4:6], dev[:0, 6:], cache.k, cache.v, none, none,
                              table.cuda())
    assert got.shape == (0, 4, 128)
    # one position for all tokens
    same = torch.tensor([3], device="cuda").expand(20)
    got = fat.kv_cache_append(dev[:, :4], dev[:, 4:6], dev[:, 6:], cache.k, cache.v, slots.cuda(),
                              same, table.cuda())
    assert torch.equal(got.cpu(), plain(q, table, torch.full((1, 20), 3), None, False).bfloat16())
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_indexes_outside_their_tensors(cuda_device, kind):
    """They are reported, and the token is neither stored nor given out."""
    cache, slots, positions, table, (q, k, v) = setup(6, 3, 2, 16, 64, "bf16", kind, "phtd", 64,
                                                      None)
    for where, bad in (("position", -1), ("position", 500), ("position", 2 ** 40),
                       ("slot", cache.k.shape[0] * 16), ("slot", 2 ** 62)):
        s, p = slots.clone(), positions[0].clone()
        (p if where == "position" else s)[4] = bad
        before = cache.held()
        out = torch.full((6, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        fat.kv_cache_append(q.cuda(), k.cuda(), v.cuda(), cache.k, cache.v, s.cuda(), p.cuda(),
                            table.cuda(), out=out, **cache.scale_args)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX
        assert fat.check_device_error() == fat.FAT_OK
        if where == "position":
            assert (out[4] == 7).all()
        good = [t for t in range(6) if t != 4]
        assert torch.equal(out[good].cpu(), plain(q, table, positions, None, False)
                           .bfloat16()[good])
        after = cache.held()
        for x, y in zip(after, before):
            for t in good:
                if slots[t] >= 0:
                    y[slots[t] // 16, :, slots[t] % 16] = x[slots[t] // 16, :, slots[t] % 16]
            assert torch.equal(x, y)


def test_rows_with_infinities_and_nan(cuda_device):
    cache, slots, positions, table, (q, k, v) = setup(8, 1, 1, 16, 64, "bf16", "e4m3", "phtd", 64,
                                                      None)
    k[0, 0, 5], k[1, 0, 40], v[3, 0, 1] = math.inf, math.nan, -math.inf
    slots[:4] = torch.tensor([0, 17, 3, 33])
    slots[4:] = torch.tensor([5, 6, 7, 8])
    fat.kv_cache_append(None, k.cuda(), v.cuda(), cache.k, cache.v, slots.cuda(),
                        positions[0].cuda(), table.cuda(), **cache.scale_args)
    kk, vv = cache.held()
    bad = [torch.isnan(x[slots // 16, 0, slots % 16]).all(-1).tolist() for x in (kk, vv)]
    assert bad[0] == [True, True] + [False] * 6 and bad[1] == [False] * 3 + [True] + [False] * 4


def test_refusals(cuda_device):
    cache, slots, positions, table, (q, k, v) = setup(6, 4, 2, 16, 64, "bf16", "bf16", "phtd", 64,
                                                      None)
    good = dict(q=q.cuda(), k=k.cuda(), v=v.cuda(), k_cache=cache.k, v_cache=cache.v,
                slots=slots.cuda(), positions=positions[0].cuda(), cos_sin=table.cuda())
    fat.kv_cache_append(**good)
    two = torch.stack([good["positions"]] * 2)
    for bad in (dict(q=q), dict(q=good["q"].half()), dict(q=good["q"][:5]),
                dict(q=good["q"][..., :32]), dict(k=good["k"].half(), v=good["v"].half()),
                dict(slots=good["slots"].int()), dict(slots=good["slots"][:5]),
                dict(slots=torch.stack([good["slots"]] * 2, 1)[:, 0]),
                dict(positions=good["positions"].int()), dict(positions=good["positions"][:5]),
                dict(positions=two), dict(positions=two, sections=(16, 15)),
                dict(positions=two, sections=(40, -8)), dict(positions=two, sections=(32,)),
                dict(positions=good["positions"], sections=(32,)),
                dict(positions=two, sections=()), dict(cos_sin=table.cuda().double()),
                dict(cos_sin=table.cuda()[:, :24]), dict(cos_sin=torch.cat([table] * 2, 1).cuda()),
                dict(cos_sin=table.cuda().T), dict(q=None, out=good["q"]),
                dict(out=good["q"][:, :2]), dict(out=good["q"].half()),
                dict(k_cache=cache.k[:1].expand(4, 2, 16, 64),
                     v_cache=cache.v[:1].expand(4, 2, 16, 64)),
                dict(k_scale=torch.zeros(cache.k.shape[:3], dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            fat.kv_cache_append(**{**good, **bad})
    odd = torch.zeros((6, 4, 72), dtype=torch.bfloat16, device="cuda")[..., 4:68]
    with pytest.raises(fat.FatError, match="ALIGNMENT"):
        fat.kv_cache_append(**{**good, "q": odd})
    with pytest.raises(fat.FatError, match="ALIGNMENT"):
        fat.kv_cache_append(**{**good, "cos_sin": torch.zeros((500, 66), device="cuda")[:, :64]})
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK


