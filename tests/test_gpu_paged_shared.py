"""Sequences that share the pages of a common prefix: bounds, scores and attention."""
import numpy as np
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import Cache, check_attention, queries, ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[64, 64, 64], [70, 64, 95, 81], [40, 40]], ids=str)
def test_shared_prefix(cuda_device, kind, lens):
    """The prefix's pages stand in every line; what follows is each sequence's own.  [40, 40]: a
    partly filled page, to the same position in both, as after a fork."""
    ps, H, G, d = 16, 2, 4, 64
    cache = Cache(24, H, ps, d, kind, seed=len(lens))
    own = min(lens) // ps if lens != [40, 40] else 3  # pages that are shared
    order = torch.randperm(24, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    table = torch.full((len(lens), 7), 2 ** 31 - 1, dtype=torch.int32)
    at = own
    for b, n in enumerate(lens):
        count = -(-n // ps)
        table[b, :own] = order[:own]
        table[b, own:count] = order[at:at + count - own]
        at += count - own
    lens_t = torch.tensor(lens, dtype=torch.int32)
    q = queries(len(lens), H * G, d, "bf16", seed=3)
    args = (table.cuda(), lens_t.cuda())
    want_bounds = ref.bounds_of(cache.k_values, table, lens, ps, 10 ** 9,
                                torch.full((24, H, 2, d), 9.0, dtype=torch.float64))
    for new in (None, 40):
        for _ in range(5):
            bounds = torch.full((24, H, 2, d), 9.0, dtype=torch.bfloat16, device="cuda")
            if new is not None:
                fat.kv_block_bounds(cache.k, *args, bounds, k_scale=cache.scales[0])
            fat.kv_block_bounds(cache.k, *args, bounds, new, k_scale=cache.scales[0])
            assert torch.equal(bounds.cpu().double(), want_bounds.to(torch.bfloat16).double())
    scores = fat.kv_block_scores(q.cuda(), bounds, *args, ps)
    scale = float(np.float32(d ** -0.5))
    whole = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, *args, **cache.scale_args)
    check_attention(*whole, *ref.decode(q.double(), cache.k_values, cache.v_values, table, lens,
                                        ps, scale), kind=kind)
    o, lse, blocks = fat.attn_decode_sparse(q.cuda(), cache.k, cache.v, *args, scores, 3,
                                            **cache.scale_args)
    *want, chosen = ref.sparse(q.double(), cache.k_values, cache.v_values, table, lens, ps,
                               scores.cpu().double(), 3, scale)
    assert torch.equal(blocks.cpu(), chosen)
    check_attention(o, lse, *want, kind=kind)
    assert fat.check_device_error() == fat.FAT_OK
