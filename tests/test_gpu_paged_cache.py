"""Writing tokens to the paged cache and reading sequences back: every value
equals the plain implementation's (powers of two as scales make the one
rounding of each code the only one), and nothing else in the cache changes."""
import math

import numpy as np
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import TYPES, Cache, make_table, pages_for, ref

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and \
        torch.equal(torch.nan_to_num(a, 0.25), torch.nan_to_num(b, 0.25))


def stored(x, kind):
    """What rows x (fp64, [..., d]) hold in a cache of this kind."""
    if kind != "e4m3":
        return x
    flat = x.reshape(-1, x.shape[-1]).numpy()
    return torch.tensor(np.stack([ref.quantise_row(r)[0] for r in flat])).reshape(x.shape)


CASES = [
    # tokens, heads, page_size, d, token type, cache type, layout
    (1, 1, 16, 128, "bf16", "e4m3", "phtd"),
    (37, 3, 16, 128, "bf16", "e4m3", "pthd"),
    (130, 2, 64, 64, "fp16", "e4m3", "kv"),
    (19, 5, 32, 64, "bf16", "bf16", "pthd"),
    (64, 8, 256, 128, "fp16", "fp16", "kv"),
    (11, 1, 1024, 64, "bf16", "e4m3", "phtd"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_write_then_read(cuda_device, case):
    T, H, ps, d, typ, kind, layout = case
    pages = -(-T // ps) + 3
    cache = Cache(pages, H, ps, d, kind, layout, seed=T)
    g = torch.Generator().manual_seed(T + d)
    # rows of different magnitude, inside one buffer with more than K and V in a token's row
    buffer = torch.randn((T, 3, H, d), generator=g) * 2.0 ** torch.randint(-9, 9, (T, 1, H, 1),
                                                                           generator=g)
    buffer = buffer.to(TYPES[typ]).cuda()
    k, v = buffer[:, 1], buffer[:, 2]
    perm = torch.randperm(pages * ps, generator=g)[:T].to(torch.int64)
    skip = torch.rand(T, generator=g) < 0.2
    slots = torch.where(skip, torch.tensor(-1 - T), perm).cuda()
    want = [x.clone() for x in cache.held()]
    for t in range(T):
        if not skip[t]:
            page, place = divmod(int(perm[t]), ps)
            for w, x in zip(want, (k, v)):
                w[page, :, place] = stored(x[t].cpu().double(), kind)
    fat.kv_cache_write(k, v, cache.k, cache.v, slots, **cache.scale_args)
    torch.cuda.synchronize()
    for got, w in zip(cache.held(), want):
        assert same(got, w)
    # read two "sequences" made of those pages back
    n = [pages // 2 * ps, (pages - pages // 2) * ps - 5]
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    width = max(pages // 2, pages - pages // 2)
    table = torch.full((2, width), 2 ** 31 - 1, dtype=torch.int32)
    table[0, :pages // 2] = ids[:pages // 2]
    table[1, :pages - pages // 2] = ids[pages // 2:]
    lens = torch.tensor(n, dtype=torch.int32)
    out_type = TYPES[typ]
    most = max(n) + 3
    out = fat.kv_cache_read(cache.k, cache.v, table.cuda(), lens.cuda(), most, dtype=out_type,
                            **cache.scale_args)
    torch.cuda.synchronize()
    for got, w in zip(out, want):
        full = torch.zeros((2, H, most, d), dtype=torch.float64)
        for b in range(2):
            full[b, :, :n[b]] = ref.gather(w, table[b], n[b], ps)
        assert same(got.cpu().double(), full.to(out_type).double())
    assert fat.check_device_error() == fat.FAT_OK


@pytest.mark.parametrize("typ,kind,d", [("bf16", "e4m3", 128), ("fp16", "e4m3", 64),
                                         ("bf16", "bf16", 128), ("fp16", "fp16", 64)])
def test_many_tokens(cuda_device, typ, kind, d):
    """Calls large enough for several rows to a thread, with ragged ends."""
    H, ps, lens = 9, 32, [4001, 17, 3333]
    pages = pages_for(lens, ps)
    cache = Cache(pages, H, ps, d, kind, "pthd", seed=d)
    table = make_table(lens, ps, pages, seed=d)
    slots = torch.cat([table[b, torch.arange(n) // ps].long() * ps + torch.arange(n) % ps
                       for b, n in enumerate(lens)])
    g = torch.Generator().manual_seed(d)
    x = torch.randn((2, len(slots), H, d), generator=g)
    x = (x * 2.0 ** torch.randint(-6, 7, (2, len(slots), H, 1), generator=g)).to(TYPES[typ])
    fat.kv_cache_write(x[0].cuda(), x[1].cuda(), cache.k, cache.v, slots.cuda(),
                       **cache.scale_args)
    out = fat.kv_cache_read(cache.k, cache.v, table.cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), 4005, dtype=TYPES[typ],
                            **cache.scale_args)
    held = ref.quantise_rows(x.double()) if kind == "e4m3" else x.double()
    for got, rows in zip(out, held):
        want = torch.zeros((3, H, 4005, d), dtype=torch.float64)
        at = 0
        for b, n in enumerate(lens):
            want[b, :, :n] = rows[at:at + n].transpose(0, 1)
            at += n
        assert torch.equal(got.cpu().double(), want.to(TYPES[typ]).double())
    assert fat.check_device_error() == fat.FAT_OK


def test_quantised_rows_at_the_edges(cuda_device):
    """Zeros, a magnitude exactly at and just above 448 times a power of two, subnormals, the
    largest values, infinities and NaN."""
    d, ps = 128, 16
    rows = torch.zeros((12, d))
    rows[1, 3] = 448.0
    rows[2, 3] = 450.0
    rows[3] = torch.linspace(-448.0, 448.0, d) / 2 ** 20
    rows[4, :2] = torch.tensor([1.0, 2.0 ** -12])       # underflows to zero inside the row
    rows[5] = 2.0 ** -130 * torch.arange(d)             # bf16 subnormals
    rows[6] = 3.0e38 * torch.linspace(-1, 1, d)
    rows[7, 5] = math.inf
    rows[8, 6] = -math.inf
    rows[9, 7] = math.nan
    rows[10] = -0.0
    rows[11] = 1.0 + 2.0 ** -5 * torch.arange(d)        # ties between codes
    k = rows.to(torch.bfloat16)[:, None]
    cache = Cache(1, 1, ps, d, "e4m3")
    slots = torch.arange(12)
    fat.kv_cache_write(k.cuda(), k.flip(0).contiguous().cuda(), cache.k, cache.v, slots.cuda(),
                       **cache.scale_args)
    torch.cuda.synchronize()
    want = stored(k.double(), "e4m3")[:, 0]
    got_k, got_v = cache.held()
    assert same(got_k[0, 0, :12], want) and same(got_v[0, 0, :12], want.flip(0))
    bytes_ = [ref.quantise_row(r)[1] for r in k[:, 0].double().numpy()]
    assert cache.scales[0][0, 0, :12].cpu().tolist() == bytes_
    # fp16 output rounds what fp16 cannot hold; bf16 holds everything but subnormal steps
    table = torch.zeros((1, 1), dtype=torch.int32).cuda()
    lens = torch.tensor([12], dtype=torch.int32).cuda()
    for typ in (torch.bfloat16, torch.float16):
        out, _ = fat.kv_cache_read(cache.k, cache.v, table, lens, 12, dtype=typ,
                                   **cache.scale_args)
        assert same(out[0, 0].cpu().double(), want.float().to(typ).double())


def test_offsets_past_32_bits(cuda_device):
    """A cache of 5 GiB a side: the last pages are written, read and attended to in place."""
    pages, H, ps, d = 42000, 8, 64, 128
    k = torch.empty((pages, H, ps, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() * 2 > 2 ** 32
    n = 100
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    slots = table[0].long()[torch.arange(n, device="cuda") // ps] * ps + \
        torch.arange(n, device="cuda") % ps
    g = torch.Generator().manual_seed(1)
    x = torch.randn((2, n, H, d), generator=g).to(torch.bfloat16)
    fat.kv_cache_write(x[0].cuda(), x[1].cuda(), k, v, slots)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    rk, rv = fat.kv_cache_read(k, v, table, lens, n)
    assert torch.equal(rk[0].cpu(), x[0].transpose(0, 1))
    assert torch.equal(rv[0].cpu(), x[1].transpose(0, 1))
    q = torch.randn((1, H, d), generator=g).to(torch.bfloat16)
    o, lse = fat.attn_decode_paged(q.cuda(), k, v, table, lens)
    s = torch.einsum("hd,nhd->hn", q[0].double(), x[0].double()) * d ** -0.5
    want = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), x[1].double())
    # half a bf16 step and 2^-12 of magnitudes below 4
    assert ((o[0].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10).all()
    del k, v, rk, rv
    torch.cuda.empty_cache()


def test_a_slot_or_page_outside_the_cache_is_skipped_and_reported(cuda_device):
    pages, H, ps, d = 3, 2, 16, 64
    cache = Cache(pages, H, ps, d, "e4m3")
    before = [x.clone() for x in cache.held()]
    x = torch.ones((3, H, d), dtype=torch.bfloat16, device="cuda")
    assert fat.check_device_error() == fat.FAT_OK
    slots = torch.tensor([pages * ps, 2 ** 62, 2 ** 40], device="cuda")
    fat.kv_cache_write(x, x, cache.k, cache.v, slots, **cache.scale_args)
    assert fat.check_device_error() == fat.FAT_ERR_INDEX
    assert fat.check_device_error() == fat.FAT_OK  # cleared
    for a, b in zip(cache.held(), before):
        assert same(a, b)
    table = torch.tensor([[0, 7], [-1, 1]], dtype=torch.int32, device="cuda")
    for lens in ([20, 20], [1000, -4]):
        fat.kv_cache_read(cache.k, cache.v, table, torch.tensor(lens, dtype=torch.int32).cuda(),
                          40, **cache.scale_args)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX, lens


def test_refusals(cuda_device):
    cache = Cache(3, 2, 16, 64, "e4m3")
    plain = Cache(3, 2, 16, 64, "bf16")
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(4, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    good = dict(k=x, v=x, k_cache=cache.k, v_cache=cache.v, slots=slots, **cache.scale_args)
    for bad in (dict(k=x.float()), dict(k=x[:3]), dict(v=x[:, :1]), dict(slots=slots.int()),
                dict(slots=slots.cpu()), dict(k_scale=None), dict(v_scale=cache.scales[1][:2]),
                dict(k_cache=cache.k[:2]), dict(k_cache=cache.k.expand(3, 2, 16, 64)[:, :, :, ::2]),
                dict(v=x.half()), dict(k_cache=plain.k),
                dict(k_cache=cache.k[:1].expand(3, 2, 16, 64))):
        with pytest.raises(ValueError):
            fat.kv_cache_write(**{**good, **bad})
    with pytest.raises(ValueError):  # a 16-bit cache takes its own type
        fat.kv_cache_write(x.half(), x.half(), plain.k, plain.v, slots)
    with pytest.raises(ValueError):  # and no scales
        fat.kv_cache_write(x, x, plain.k, plain.v, slots, **cache.scale_args)
    odd = torch.ones((4, 2, 65), dtype=torch.bfloat16, device="cuda")[:, :, 1:]
    with pytest.raises(fat.FatError, match="ALIGNMENT"):
        fat.kv_cache_write(odd, odd, plain.k, plain.v, slots)
    for shape in ((3, 2, 24, 64), (3, 2, 8, 64), (3, 2, 16, 96)):
        k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        y = torch.zeros((4, 2, shape[3]), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(fat.FatError, match="INVALID_ARG"):
            fat.kv_cache_write(y, y, k, k.clone(), slots)
    for bad in (dict(max_len=0), dict(dtype=torch.float32), dict(dtype=torch.float16)):
        with pytest.raises(ValueError):
            fat.kv_cache_read(**{**dict(k_cache=plain.k, v_cache=plain.v, page_table=table,
                                        seq_lens=lens, max_len=4), **bad})
    with pytest.raises(ValueError):
        fat.kv_cache_read(plain.k, plain.v, table.long(), lens, 4)
    with pytest.raises(ValueError):
        fat.kv_cache_read(plain.k, plain.v, table, lens.repeat(2), 4)
    # no tokens: nothing to do
    fat.kv_cache_write(x[:0], x[:0], plain.k, plain.v, slots[:0])


def test_read_of_part_of_a_sequence_into_given_tensors(cuda_device):
    """Positions from max_len on are left out; rows of a shorter sequence are zeros."""
    lens, ps = [100, 7, 0], 16
    cache = Cache(pages_for(lens, ps), 2, ps, 64, "fp16", "pthd", seed=3)
    table = make_table(lens, ps, cache.k.shape[0], seed=3)
    out = tuple(torch.full((3, 2, 33, 64), 9.0, dtype=torch.float16, device="cuda")
                for _ in range(2))
    got = fat.kv_cache_read(cache.k, cache.v, table.cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), 33, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for t, values in zip(out, cache.values):
        want = torch.zeros((3, 2, 33, 64), dtype=torch.float64)
        for b, n in enumerate(lens):
            want[b, :, :min(n, 33)] = ref.gather(values, table[b], min(n, 33), ps)
        assert torch.equal(t.cpu().double(), want)
    assert fat.check_device_error() == fat.FAT_OK


def test_write_and_read_on_another_stream(cuda_device):
    cache = Cache(pages_for([50], 16), 2, 16, 128, "bf16")
    x = torch.randn((50, 2, 128), device="cuda").to(torch.bfloat16)
    table = make_table([50], 16, cache.k.shape[0]).cuda()
    at = torch.arange(50, device="cuda")
    slots = table[0].long()[at // 16] * 16 + at % 16
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fat.kv_cache_write(x, x, cache.k, cache.v, slots, stream=s)
    k, v = fat.kv_cache_read(cache.k, cache.v, table, lens, 50, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(k[0], x.transpose(0, 1)) and torch.equal(v, k)
