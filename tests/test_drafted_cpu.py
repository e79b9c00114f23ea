"""The C entry points of a step of drafted tokens, and of windowed attention, refuse bad arguments
before anything is launched; masks of trees; the walk over what a window sees, as the kernels
compute it, on the host."""
import ctypes
import math
import random
import subprocess

import pytest
import torch

import drafted_reference
import tensorized_online_softmax_gb300 as fat
from tensorized_online_softmax_gb300 import _build, drafted
from tensorized_online_softmax_gb300.drafted import FatRotation
from test_paged_cpu import (BAD_CACHES, BAD_QUERIES, BAD_TABLES, BAD_V, BF16, E4M3, FP16, REACHED,
                            cache, lib, refused, table)

assert lib  # (the fixture)


def rotation(**kw):
    r = dict(cos_sin=0x500000, rows=100, row_stride=128, positions=0x600000, axis_stride=5,
             token_stride=1, dim=128, axes=1, sections=(0, 0, 0, 0), interleaved=0)
    r.update(kw)
    r["sections"] = (ctypes.c_int * 4)(*r["sections"])
    return ctypes.byref(FatRotation(**r))


def append(lib, c=None, r=None, q=0x400000, qs=(512, 128), q_heads=4, k=0x100000, v=0x200000,
           dtype=BF16, ks=(256, 128), vs=(256, 128), slots=0x300000, tokens=5, out=0x700000):
    return lib.fat_kv_append(c or cache(), r or rotation(), q, *qs, q_heads, k, v, dtype, *ks, *vs,
                             slots, tokens, out, None)


def window(lib, c=None, t=None, q=0x70000, dtype=BF16, batch_stride=1024, head_stride=128,
           q_heads=8, window=1000, sinks=4, scale=0.1, o=0x80000, lse=0x90000, work=0xA0000,
           size=1 << 30):
    return lib.fat_attn_decode_window(c or cache(), t or table(), q, dtype, batch_stride,
                                      head_stride, q_heads, window, sinks, scale, o, lse, work,
                                      size, None)


def tree(lib, c=None, t=None, q=0x70000, dtype=BF16, batch_stride=1 << 13, token_stride=1024,
         head_stride=128, q_heads=8, tokens=8, masks=0xB0000, tree_stride=8, draft_lens=0xC0000,
         window=0, sinks=0, scale=0.1, o=0x80000, lse=0x90000, work=0xA0000, size=1 << 40):
    return lib.fat_attn_tree_paged(c or cache(), t or table(), q, dtype, batch_stride,
                                   token_stride, head_stride, q_heads, tokens, masks, tree_stride,
                                   draft_lens, window, sinks, scale, o, lse, work, size, None)


def keep(lib, c=None, t=None, path=0xB0000, stride=8, width=8, counts=0xC0000):
    return lib.fat_kv_keep(c or cache(), t or table(), path, stride, width, counts, None)


def test_good_arguments_reach_the_device_check(lib):
    for call in (append, window, tree, keep):
        assert call(lib) in REACHED, call.__name__
    e4m3 = cache(dtype=E4M3)
    for call in (append, window, tree):
        assert call(lib, c=e4m3, dtype=FP16) in REACHED, call.__name__
    assert keep(lib, c=e4m3) in REACHED
    assert append(lib, tokens=0, k=None) == fat.FAT_OK
    assert append(lib, q=None, out=None, q_heads=0) in REACHED
    assert append(lib, r=rotation(axes=3, sections=(16, 24, 24, 0), dim=128)) in REACHED
    assert append(lib, r=rotation(axes=4, sections=(0, 0, 8, 0), dim=16)) in REACHED
    assert append(lib, r=rotation(dim=32, interleaved=1)) in REACHED
    assert tree(lib, draft_lens=None, tree_stride=0, window=8, sinks=1) in REACHED
    # 32 pages of 16 positions, or a window and sinks of 7 tiles of 64: nothing is split
    assert window(lib, t=table(width=32), work=None, size=0) in REACHED
    assert window(lib, window=385 - 64 + 63, sinks=64, work=None, size=0) in REACHED
    refused(window(lib, window=385, sinks=64, work=None, size=0), "INVALID_ARG")


@pytest.mark.parametrize("kw,name", BAD_CACHES + BAD_V, ids=str)
def test_bad_caches(lib, kw, name):
    for call in (append, window, tree, keep):
        refused(call(lib, c=cache(**kw)), name)


@pytest.mark.parametrize("kw,name", BAD_TABLES, ids=str)
def test_bad_tables(lib, kw, name):
    for call in (window, tree, keep):
        refused(call(lib, t=table(**kw)), name)


@pytest.mark.parametrize("kw,name", BAD_QUERIES, ids=str)
def test_bad_queries(lib, kw, name):
    for call in (window, tree):
        refused(call(lib, **kw), name)


@pytest.mark.parametrize("call,kw,name", [
    (append, dict(k=None), "INVALID_ARG"), (append, dict(slots=None), "INVALID_ARG"),
    (append, dict(q=None), "INVALID_ARG"), (append, dict(out=None), "INVALID_ARG"),
    (append, dict(q_heads=-1), "INVALID_ARG"), (append, dict(tokens=-1), "INVALID_ARG"),
    (append, dict(dtype=FP16), "INVALID_ARG"), (append, dict(dtype=E4M3), "INVALID_ARG"),
    (append, dict(tokens=2 ** 31 - 1), "INVALID_ARG"),
    (append, dict(q_heads=2 ** 31 - 1), "INVALID_ARG"),
    (append, dict(qs=(513, 128)), "ALIGNMENT"), (append, dict(ks=(256, 4)), "ALIGNMENT"),
    (append, dict(q=0x400008), "ALIGNMENT"), (append, dict(out=0x700008), "ALIGNMENT"),
    (append, dict(slots=0x300004), "ALIGNMENT"),
    (window, dict(window=0), "INVALID_ARG"), (window, dict(window=-1), "INVALID_ARG"),
    (window, dict(sinks=-1), "INVALID_ARG"), (window, dict(dtype=FP16), "INVALID_ARG"),
    (window, dict(work=None), "INVALID_ARG"), (window, dict(size=8), "INVALID_ARG"),
    (window, dict(scale=-1.0), "INVALID_ARG"), (window, dict(o=None), "INVALID_ARG"),
    (window, dict(o=0x80008), "ALIGNMENT"), (window, dict(work=0xA0004), "ALIGNMENT"),
    (tree, dict(tokens=0), "INVALID_ARG"), (tree, dict(tokens=65), "INVALID_ARG"),
    (tree, dict(masks=None), "INVALID_ARG"), (tree, dict(tree_stride=-1), "INVALID_ARG"),
    (tree, dict(window=7), "INVALID_ARG"), (tree, dict(window=-1), "INVALID_ARG"),
    (tree, dict(sinks=-1), "INVALID_ARG"), (tree, dict(dtype=FP16), "INVALID_ARG"),
    (tree, dict(scale=math.nan), "INVALID_ARG"), (tree, dict(o=None), "INVALID_ARG"),
    (tree, dict(lse=None), "INVALID_ARG"), (tree, dict(work=None), "INVALID_ARG"),
    (tree, dict(size=8), "INVALID_ARG"), (tree, dict(token_stride=1028), "ALIGNMENT"),
    (tree, dict(masks=0xB0004), "ALIGNMENT"), (tree, dict(draft_lens=0xC0002), "ALIGNMENT"),
    (tree, dict(work=0xA0008), "ALIGNMENT"), (tree, dict(o=0x80008), "ALIGNMENT"),
    (tree, dict(lse=0x90002), "ALIGNMENT"),
    (tree, dict(scale=3e38), "INVALID_ARG"),  # times log2(e) fp32 does not hold it
    (tree, dict(head_stride=0), "UNSUPPORTED"), (tree, dict(token_stride=0), "UNSUPPORTED"),
    (tree, dict(c=cache(k_token_stride=0)), "UNSUPPORTED"),
    (tree, dict(c=cache(v_token_stride=0)), "UNSUPPORTED"),
    (keep, dict(path=None), "INVALID_ARG"), (keep, dict(counts=None), "INVALID_ARG"),
    (keep, dict(width=0), "INVALID_ARG"), (keep, dict(stride=-1), "INVALID_ARG"),
    (keep, dict(path=0xB0002), "ALIGNMENT"), (keep, dict(counts=0xC0002), "ALIGNMENT"),
], ids=lambda x: getattr(x, "__name__", str(x)))
def test_bad_arguments(lib, call, kw, name):
    refused(call(lib, **kw), name)


@pytest.mark.parametrize("kw,name", [
    (dict(cos_sin=None), "INVALID_ARG"), (dict(positions=None), "INVALID_ARG"),
    (dict(rows=0), "INVALID_ARG"), (dict(row_stride=124), "INVALID_ARG"),
    (dict(dim=0), "INVALID_ARG"), (dict(dim=24), "INVALID_ARG"), (dict(dim=144), "INVALID_ARG"),
    (dict(axes=0), "INVALID_ARG"), (dict(axes=5), "INVALID_ARG"),
    (dict(axes=3, sections=(16, 24, 23, 0)), "INVALID_ARG"),
    (dict(axes=3, sections=(16, 24, 25, 0)), "INVALID_ARG"),
    (dict(axes=2, sections=(65, -1, 0, 0)), "INVALID_ARG"),
    (dict(axes=2, sections=(2 ** 31 - 1, 2 ** 31 - 1, 0, 0)), "INVALID_ARG"),
    (dict(axes=2, sections=(32, 32, 0, 0), axis_stride=-1), "INVALID_ARG"),
    (dict(token_stride=-1), "INVALID_ARG"), (dict(positions=0x600004), "ALIGNMENT"),
    (dict(cos_sin=0x500008), "ALIGNMENT"), (dict(row_stride=130), "ALIGNMENT"),
], ids=str)
def test_bad_rotations(lib, kw, name):
    refused(append(lib, r=rotation(**kw)), name)


def test_no_rotation_is_refused(lib):
    assert lib.fat_kv_append(cache(), None, 0x400000, 512, 128, 4, 0x100000, 0x200000, BF16, 256,
                             128, 256, 128, 0x300000, 5, 0x700000, None) == fat.FAT_ERR_INVALID_ARG


def test_workspace_sizes(lib):
    assert lib.fat_attn_tree_workspace_bytes(3, 8, 8, 2, 128) > 0
    for bad in ((0, 8, 8, 2, 128), (3, 0, 8, 2, 128), (3, 65, 8, 2, 128), (3, 8, 7, 2, 128),
                (3, 8, 8, 0, 128), (3, 8, 8, 2, 96), (2 ** 31 - 1, 8, 8, 2, 128)):
        assert lib.fat_attn_tree_workspace_bytes(*bad) == 0


def test_struct_layout():
    values = (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13)
    r = FatRotation(*values[:8], (ctypes.c_int * 4)(*values[8:12]), values[12])
    assert bytes(r) == drafted._pack_rotation(*values)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fat.attn_tree_paged(x, x, x, t, n, torch.ones(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        fat.attn_decode_window(x[:, :, 0], x, x, t, n, 5)
    with pytest.raises(ValueError, match="CUDA"):
        fat.kv_cache_append(None, x[:, 0], x[:, 0], x, x, n, n, x)
    with pytest.raises(ValueError, match="CUDA"):
        fat.kv_cache_keep(x, x, t, n, t, n)


# ------------------------------------------------------------- masks of trees
def test_tree_mask():
    parents = torch.tensor([-1, 0, 0, 1, -1, 4])
    assert fat.tree_mask(parents).tolist() == [1, 3, 5, 11, 16, 48]
    chain = torch.arange(-1, 63)
    want = [2 ** (t + 1) - 1 for t in range(64)]
    assert [x % 2 ** 64 for x in fat.tree_mask(chain).tolist()] == want
    both = torch.stack([parents, torch.tensor([-1, -1, 1, 2, 3, 0])]).to(torch.int32)
    assert fat.tree_mask(both).tolist() == [[1, 3, 5, 11, 16, 48], [1, 2, 6, 14, 30, 33]]
    # what is no earlier token is none
    assert fat.tree_mask(torch.tensor([0, 5, -7])).tolist() == [1, 2, 4]
    for bad in (torch.zeros(65, dtype=torch.int64), torch.zeros(0, dtype=torch.int64),
                torch.zeros(3), torch.tensor(1)):
        with pytest.raises(ValueError):
            fat.tree_mask(bad)


# ------------------------------------------------- the walk over what is seen
PROGRAM = r"""
#include <cstdio>
#include "fat_decode_plan.h"
int main() {
  int len, window, sinks, tile;
  while (std::scanf("%d %d %d %d", &len, &window, &sinks, &tile) == 4) {
    const fat::DecodeSpan s = fat::decode_span(len, window, sinks, tile);
    std::printf("%d %lld", s.tiles, fat::decode_span_most(len, window, sinks, tile));
    for (int i = 0; i < s.tiles; ++i) std::printf(" %d", fat::decode_span_tile(s, i));
    std::printf(";");
    for (int j = 0; j < len && len < 5000; ++j)
      std::printf("%d", fat::decode_span_sees(s, j) ? 1 : 0);
    std::printf("\n");
  }
}
"""


def test_the_walk_over_a_window(tmp_path):
    source = tmp_path / "walk.cpp"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", _build.CSRC, "-o", str(tmp_path / "walk"),
                    str(source)], check=True)
    rng = random.Random(4)
    cases = [(n, w, s, tile) for n in (0, 1, 63, 64, 65, 200, 640, 700) for w in (1, 64, 65, 300)
             for s in (0, 1, 64, 70, 500) for tile in (64, 128)]
    cases += [(rng.randint(0, 3000), rng.randint(1, 1500), rng.randint(0, 300), 64)
              for _ in range(200)]
    cases += [(900, 0, 0, 64), (2 ** 30, 2 ** 30, 7, 64), (2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1, 128),
              (2 ** 30, 100, 100, 64)]
    out = subprocess.run([str(tmp_path / "walk")], text=True, capture_output=True, check=True,
                         input="".join("%d %d %d %d\n" % c for c in cases if c[0] < 5000 or
                                       c[1] < 1000))
    lines = iter(out.stdout.splitlines())
    for n, w, s, tile in cases:
        if n >= 5000 and w >= 1000:
            continue  # (too many tiles to print)
        head, bits = next(lines).split(";")
        tiles, most, *walk = map(int, head.split())
        want = {j // tile for j in range(n) if not w or j < s or j >= n - w} if n < 5000 else \
            {j // tile for j in list(range(s)) + list(range(n - w, n))}
        assert walk == sorted(want) if want else walk == [0], (n, w, s, tile)
        assert tiles == len(walk) <= most, (n, w, s, tile)
        if n < 5000:
            assert bits == "".join("1" if not w or j < s or j >= n - w else "0"
                                   for j in range(n)), (n, w, s, tile)


def test_reference_of_a_chain_is_decode_with_growing_lengths():
    import paged_reference as ref
    g = torch.Generator().manual_seed(0)
    k, v = torch.randn((2, 7, 2, 16, 64), generator=g, dtype=torch.float64)
    q = torch.randn((1, 3, 4, 64), generator=g, dtype=torch.float64)
    t = torch.tensor([[3, 1, 6]])
    o, lse, _ = drafted_reference.tree(q, k, v, t, [40], [3], [[1, 3, 7]], 16, 0.125)
    for i in range(3):
        want = ref.decode(q[:, i], k, v, t, [38 + i], 16, 0.125)
        assert torch.allclose(o[:, i], want[0], atol=1e-14)
        assert torch.allclose(lse[:, i], want[1], atol=1e-14)
    o, lse, _ = drafted_reference.window(q[:, 0], k, v, t, [40], 16, 0.125, 7, 2)
    at = [0, 1] + list(range(33, 40))
    kk, vv = (torch.cat([x[3, 1], x[1, 1], x[6, 1]])[at] for x in (k, v))
    e = torch.exp(kk @ q[0, 0, 3] * 0.125)
    assert torch.allclose(o[0, 3], (e[:, None] * vv).sum(0) / e.sum(), atol=1e-12)
