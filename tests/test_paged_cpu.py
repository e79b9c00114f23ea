"""The paged cache's C entry points refuse bad arguments before anything is
launched (no GPU here: a call that passes the checks ends with the device
check), and the plain 64-bit implementation used by the GPU tests agrees with
independent forms of the same definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_reference as ref
import tensorized_online_softmax_gb300 as fat
from tensorized_online_softmax_gb300 import paged
from tensorized_online_softmax_gb300.paged import FatKvCache, FatPageTable

BF16, E4M3, FP16 = 0, 1, 2
REACHED = (fat.FAT_ERR_LAUNCH, fat.FAT_ERR_ARCH)  # past the checks, on a host without the GPU


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for hosts without a GPU")
    return fat.load_library()


def cache(**kw):
    c = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, num_pages=10, heads=2,
             page_size=16, d=128, dtype=BF16, k_page_stride=4096, k_head_stride=2048,
             k_token_stride=128, v_page_stride=4096, v_head_stride=2048, v_token_stride=128)
    return ctypes.byref(FatKvCache(**{**c, **kw}))


def table(**kw):
    # (room for 1024 positions: more than a call without workspace takes)
    return ctypes.byref(FatPageTable(**{**dict(pages=0x50000, stride=64, width=64, batch=3,
                                               seq_lens=0x60000), **kw}))


BAD_CACHES = [
    (dict(k=None), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(num_pages=1 << 31), "INVALID_ARG"), (dict(heads=0), "INVALID_ARG"),
    (dict(page_size=0), "INVALID_ARG"), (dict(page_size=8), "INVALID_ARG"),
    (dict(page_size=48), "INVALID_ARG"), (dict(page_size=2048), "INVALID_ARG"),
    (dict(d=96), "INVALID_ARG"), (dict(dtype=3), "INVALID_ARG"), (dict(dtype=-1), "INVALID_ARG"),
    (dict(dtype=E4M3, k_scale=None), "INVALID_ARG"), (dict(k=0x10008), "ALIGNMENT"),
    (dict(k_token_stride=132), "ALIGNMENT"), (dict(k_page_stride=1 << 31), "ALIGNMENT"),
    (dict(k_head_stride=-2048), "ALIGNMENT"),
    (dict(dtype=E4M3, k_page_stride=4104), "ALIGNMENT"),
    (dict(dtype=E4M3, k_scale=0x30008), "ALIGNMENT"),
]
BAD_V = [(dict(v=None), "INVALID_ARG"), (dict(v=0x20004), "ALIGNMENT"),
         (dict(v_page_stride=4), "ALIGNMENT"), (dict(dtype=E4M3, v_scale=None), "INVALID_ARG")]
BAD_TABLES = [(dict(pages=None), "INVALID_ARG"), (dict(seq_lens=None), "INVALID_ARG"),
              (dict(width=0), "INVALID_ARG"), (dict(batch=0), "INVALID_ARG"),
              (dict(stride=63), "INVALID_ARG"),
              (dict(stride=1 << 28, width=(1 << 26) + 1), "INVALID_ARG"), (dict(pages=0x50002), "ALIGNMENT"),
              (dict(seq_lens=0x60001), "ALIGNMENT")]
BAD_QUERIES = [(dict(q=None), "INVALID_ARG"), (dict(q=0x70008), "ALIGNMENT"),
               (dict(dtype=E4M3), "INVALID_ARG"), (dict(batch_stride=1028), "ALIGNMENT"),
               (dict(head_stride=-128), "ALIGNMENT"), (dict(q_heads=0), "INVALID_ARG"),
               (dict(q_heads=7), "INVALID_ARG")]


def write(lib, c=None, k=0x100000, v=0x200000, dtype=BF16, ks=(256, 128), vs=(256, 128),
          slots=0x300000, tokens=5):
    return lib.fat_kv_write(c or cache(), k, v, dtype, *ks, *vs, slots, tokens, None)


def read(lib, c=None, t=None, k=0x100000, v=0x200000, dtype=BF16, max_len=9):
    return lib.fat_kv_read(c or cache(), t or table(), k, v, dtype, max_len, None)


def decode(lib, c=None, t=None, q=0x70000, dtype=BF16, batch_stride=1024, head_stride=128,
           q_heads=8, scale=0.1, o=0x80000, lse=0x90000, work=0xA0000, size=1 << 30):
    return lib.fat_attn_decode_paged(c or cache(), t or table(), q, dtype, batch_stride,
                                     head_stride, q_heads, scale, o, lse, work, size, None)


def sparse(lib, c=None, t=None, q=0x70000, dtype=BF16, batch_stride=1024, head_stride=128,
           q_heads=8, scores=0xB0000, num_blocks=4, first=0, last=1, scale=0.1, o=0x80000,
           lse=0x90000, blocks=0xC0000, work=0xA0000, size=1 << 30):
    return lib.fat_attn_decode_sparse(c or cache(), t or table(), q, dtype, batch_stride,
                                      head_stride, q_heads, scores, num_blocks, first, last,
                                      scale, o, lse, blocks, work, size, None)


def bounds(lib, c=None, t=None, new=1, out=0xD0000, dtype=BF16):
    return lib.fat_kv_block_bounds(c or cache(), t or table(), new, out, dtype, None)


def scores(lib, t=None, q=0x70000, dtype=BF16, batch_stride=1024, head_stride=128, q_heads=8,
           b=0xD0000, pages=10, heads=2, page_size=16, d=128, out=0xB0000):
    return lib.fat_kv_block_scores(q, dtype, batch_stride, head_stride, q_heads, b, pages, heads,
                                   page_size, d, t or table(), out, None)


def refused(status, name):
    assert fat.status_string(status) == "FAT_ERR_" + name


def test_good_arguments_reach_the_device_check(lib):
    for call in (write, read, decode, sparse, bounds, scores):
        assert call(lib) in REACHED, call.__name__
    e4m3 = cache(dtype=E4M3)
    for call in (write, read, decode, sparse, bounds):
        assert call(lib, c=e4m3, dtype=FP16) in REACHED, call.__name__
    assert bounds(lib, c=cache(v=None)) in REACHED
    assert write(lib, tokens=0) == fat.FAT_OK
    # 32 pages of 16 positions: no sequence is split, and no workspace is needed
    assert decode(lib, t=table(width=32), work=None, size=0) in REACHED
    refused(decode(lib, t=table(width=33), work=None, size=0), "INVALID_ARG")


@pytest.mark.parametrize("kw,name", BAD_CACHES, ids=str)
def test_bad_caches(lib, kw, name):
    for call in (write, read, decode, sparse, bounds):
        refused(call(lib, c=cache(**kw)), name)


@pytest.mark.parametrize("kw,name", BAD_V, ids=str)
def test_bad_values(lib, kw, name):
    for call in (write, read, decode, sparse):
        refused(call(lib, c=cache(**kw)), name)


@pytest.mark.parametrize("kw,name", BAD_TABLES, ids=str)
def test_bad_tables(lib, kw, name):
    for call in (read, decode, sparse, bounds, scores):
        refused(call(lib, t=table(**kw)), name)


@pytest.mark.parametrize("kw,name", BAD_QUERIES, ids=str)
def test_bad_queries(lib, kw, name):
    for call in (decode, sparse, scores):
        refused(call(lib, **kw), name)


@pytest.mark.parametrize("call,kw,name", [
    (write, dict(k=None), "INVALID_ARG"), (write, dict(slots=None), "INVALID_ARG"),
    (write, dict(tokens=-1), "INVALID_ARG"), (write, dict(dtype=FP16), "INVALID_ARG"),
    (write, dict(dtype=E4M3), "INVALID_ARG"), (write, dict(ks=(257, 128)), "ALIGNMENT"),
    (write, dict(slots=0x300004), "ALIGNMENT"), (read, dict(max_len=0), "INVALID_ARG"),
    (read, dict(dtype=FP16), "INVALID_ARG"), (read, dict(v=None), "INVALID_ARG"),
    (read, dict(k=0x100002), "ALIGNMENT"), (decode, dict(dtype=FP16), "INVALID_ARG"),
    (decode, dict(scale=0.0), "INVALID_ARG"), (decode, dict(scale=math.inf), "INVALID_ARG"),
    (decode, dict(o=None), "INVALID_ARG"), (decode, dict(lse=None), "INVALID_ARG"),
    (decode, dict(work=None), "INVALID_ARG"), (decode, dict(size=8), "INVALID_ARG"),
    (decode, dict(work=0xA0004), "ALIGNMENT"), (decode, dict(o=0x80008), "ALIGNMENT"),
    (sparse, dict(num_blocks=0), "INVALID_ARG"), (sparse, dict(first=4), "INVALID_ARG"),
    (sparse, dict(last=5), "INVALID_ARG"), (sparse, dict(first=-1), "INVALID_ARG"),
    (sparse, dict(scores=None), "INVALID_ARG"), (sparse, dict(blocks=None), "INVALID_ARG"),
    (sparse, dict(first=2 ** 31 - 1, last=2 ** 31 - 1), "INVALID_ARG"),
    (bounds, dict(new=0), "INVALID_ARG"), (bounds, dict(out=None), "INVALID_ARG"),
    (bounds, dict(dtype=FP16), "INVALID_ARG"), (bounds, dict(out=0xD0008), "ALIGNMENT"),
    (scores, dict(b=None), "INVALID_ARG"), (scores, dict(out=None), "INVALID_ARG"),
    (scores, dict(pages=0), "INVALID_ARG"), (scores, dict(page_size=17), "INVALID_ARG"),
    (scores, dict(d=256), "INVALID_ARG"), (scores, dict(heads=3), "INVALID_ARG"),
    (scores, dict(b=0xD0004), "ALIGNMENT"),
], ids=lambda x: getattr(x, "__name__", str(x)))
def test_bad_arguments(lib, call, kw, name):
    refused(call(lib, **kw), name)


def test_workspace_sizes(lib):
    assert lib.fat_attn_decode_workspace_bytes(3, 8, 2, 128) > 0
    assert lib.fat_attn_decode_sparse_workspace_bytes(3, 8, 2, 128, 64) >= \
        lib.fat_attn_decode_workspace_bytes(3, 8, 2, 128) + 3 * 2 * 65 * 4
    for bad in ((0, 8, 2, 128), (3, 7, 2, 128), (3, 8, 0, 128), (3, 8, 2, 96)):
        assert lib.fat_attn_decode_workspace_bytes(*bad) == 0
        assert lib.fat_attn_decode_sparse_workspace_bytes(*bad, 4) == 0
    assert lib.fat_attn_decode_sparse_workspace_bytes(3, 8, 2, 128, 0) == 0
    assert lib.fat_attn_decode_sparse_workspace_bytes(3, 8, 2, 128, 2 ** 31 - 1) == 0
    assert lib.fat_attn_decode_workspace_bytes(2 ** 31 - 1, 8, 2, 128) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fat.attn_decode_paged(x[:, :, 0], x, x, torch.zeros((2, 1), dtype=torch.int32),
                              torch.zeros(2, dtype=torch.int32))


# ------------------------------------------------- the plain implementation
def test_reference_rounding_equals_the_type():
    """round_e4m3 against torch's own conversion, over all halves between codes and random values."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    middle = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, middle, middle * (1 + 1e-6), middle * (1 - 1e-6),
                   torch.randn(2000, dtype=torch.float64) * 50]).clamp(-448, 448)
    x = x.float().double()
    assert torch.equal(torch.tensor(ref.round_e4m3(x.numpy())),
                       x.float().to(torch.float8_e4m3fn).double())


def test_reference_rows_at_once():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((40, 64), generator=g, dtype=torch.float64)
    x = (x * 2.0 ** torch.randint(-40, 40, (40, 1), generator=g)).to(torch.bfloat16).double()
    x[5] = 0
    want = np.stack([ref.quantise_row(r)[0] for r in x.numpy()])
    assert torch.equal(ref.quantise_rows(x), torch.tensor(want))


def test_reference_scale_is_the_least():
    for top in (448.0, 448.1, 449.0, 1.75, 1.7500001, 3e38, 1e-30, 2.0 ** -133):
        values, e = ref.quantise_row(np.array([top, -top / 3]))
        assert top <= 448 * 2.0 ** (e - 127) and (e == 1 or top > 448 * 2.0 ** (e - 128))
        assert abs(values[0] - top) <= max(top / 16, 2.0 ** -136)


def test_reference_sparse_with_all_blocks_is_decode():
    g = torch.Generator().manual_seed(0)
    k, v = torch.randn((2, 7, 2, 16, 64), generator=g, dtype=torch.float64)
    q = torch.randn((2, 4, 64), generator=g, dtype=torch.float64)
    t = torch.tensor([[3, 1, 6], [0, 2, 5]])
    lens = [40, 33]
    o, lse, _ = ref.decode(q, k, v, t, lens, 16, 0.125)
    o2, lse2, _, blocks = ref.sparse(q, k, v, t, lens, 16, torch.zeros((2, 2, 3)), 3, 0.125)
    assert torch.allclose(o, o2, atol=1e-14) and torch.allclose(lse, lse2, atol=1e-14)
    assert blocks.tolist() == [[[0, 1, 2]] * 2] * 2
    # and one head written out
    kk = torch.cat([k[3, 1], k[1, 1], k[6, 1]])[:40]
    vv = torch.cat([v[3, 1], v[1, 1], v[6, 1]])[:40]
    e = torch.exp(kk @ q[0, 3] * 0.125)
    assert torch.allclose(o[0, 3], (e[:, None] * vv).sum(0) / e.sum(), atol=1e-12)
    assert math.isclose(lse[0, 3].item(), math.log(e.sum().item()), rel_tol=1e-12)


def test_struct_sizes():
    """The structs' layouts: 4 pointers, a 64-bit count, 4 ints, 6 strides; and the table's."""
    assert ctypes.sizeof(FatKvCache) == 4 * 8 + 8 + 4 * 4 + 6 * 8
    assert ctypes.sizeof(FatPageTable) == 8 + 8 + 4 + 4 + 8
    c = FatKvCache(*range(1, 16))
    assert bytes(c) == paged._pack_cache(*range(1, 16))
    assert bytes(FatPageTable(1, 2, 3, 4, 5)) == paged._pack_table(1, 2, 3, 4, 5)
