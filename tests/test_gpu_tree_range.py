"""Attention of drafted tokens, and of single ones, over values near the largest that it takes: the
largest magnitude times the positions that a row sees just below 2^120 over a bf16 cache, 2^113 over
an e4m3 one."""
import math

import numpy as np
import pytest
import torch

import drafted_reference
import tensorized_online_softmax_gb300 as fat
from drafted_helpers import as_tensor, check_tree
from paged_helpers import Cache, check_attention, make_table, pages_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [0, 3400], ids=["table", "long_table"])
@pytest.mark.parametrize("signs", [False, True], ids=["one_sign", "both_signs"])
@pytest.mark.parametrize("kind,T,group,d", [("bf16", 4, 2, 64), ("bf16", 60, 4, 128),
                                            ("e4m3", 4, 2, 128), ("e4m3", 40, 3, 64)])
def test_values_up_to_the_headroom(cuda_device, kind, T, group, d, signs, more):
    """The first two tiles of 128 score 0, so that each group of rows takes its reference there; all
    that follows scores nearly as much higher as a reference lets pass (8 binades, or 4): weights
    are as large as they become, and nearly all of them are.  A value is 0.9 of what the positions
    of the sequence allow."""
    page_size, n = 64, 900
    g = torch.Generator().manual_seed(T)
    cache = Cache(pages_for([n], page_size), 1, page_size, d, "bf16", seed=1)
    width = -(-n // page_size) + -(-more // page_size)
    table = make_table([n], page_size, cache.k.shape[0], seed=1, width=width)
    binades, limit = (7.8, 120) if kind == "bf16" else (3.8, 113)
    u = torch.sign(torch.randn(d, generator=g))
    k = torch.zeros((n, 1, d))
    k[256:, 0] = u * (binades * math.log(2) / math.sqrt(d))  # scale = 1 / sqrt(d), queries u
    top = 0.9 * 2.0 ** limit / n
    v = torch.full((n, 1, d), top)
    if signs:
        v *= torch.sign(torch.randn((n, 1, d), generator=g))
    scales = {}
    if kind == "e4m3":
        shape = cache.k.shape
        kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                  for _ in range(2))
        scales = {x: torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda")
                  for x in ("k_scale", "v_scale")}
    else:
        kc, vc = cache.k, cache.v
    at = torch.arange(n)
    slots = table[0, at // page_size].long() * page_size + at % page_size
    fat.kv_cache_write(k.bfloat16().cuda(), v.bfloat16().cuda(), kc, vc, slots.cuda(), **scales)
    q = u.expand(1, T, group, d).bfloat16()
    masks = [[(1 << t + 1) - 1 for t in range(T)]]
    o, lse = fat.attn_tree_paged(q.cuda(), kc, vc, table.cuda(),
                                 torch.tensor([n], dtype=torch.int32).cuda(),
                                 as_tensor(masks).cuda(), **scales)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK

    def held(x, name):
        x = x.cpu().double()
        return x if not scales else x * 2.0 ** (scales[name].cpu().double() - 127)[..., None]
    kk, vv = held(kc, "k_scale"), held(vc, "v_scale")
    assert 0.4 * 2.0 ** limit < n * vv[table[0, 5].long()].abs().max() < 2.0 ** limit
    scale = float(np.float32(d ** -0.5))
    want = drafted_reference.tree(q.double(), kk, vv, table, [n], [T], masks, page_size, scale)
    check_tree(o, lse, *want, what=f"{kind} {T} {group} {d}")
    if kind == "bf16":  # single tokens: the same headroom
        lens = torch.tensor([n], dtype=torch.int32).cuda()
        for got, window in ((fat.attn_decode_paged(q[:, 0].cuda(), kc, vc, table.cuda(), lens), n),
                            (fat.attn_decode_window(q[:, 0].cuda(), kc, vc, table.cuda(), lens,
                                                    800, 20), 800)):
            want = drafted_reference.window(q[:, 0].double(), kk, vv, table, [n], page_size, scale,
                                            window, 20)
            check_attention(*got, *want, what=f"window {window}")
