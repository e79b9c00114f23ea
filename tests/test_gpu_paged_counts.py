"""Counts beyond 32 bits are refused, not cut to what is left of them."""
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import Cache, make_table, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [2 ** 32, 2 ** 31, 2 ** 40])
def test_counts_beyond_32_bits(cuda_device, more):
    cache = Cache(5, 2, 16, 64, "bf16")
    table = make_table([40], 16, 5).cuda()
    lens = torch.tensor([40], dtype=torch.int32).cuda()
    q = queries(1, 4, 64, "bf16").cuda()
    bounds = torch.zeros((5, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros((1, 2, table.shape[1]), device="cuda")
    with pytest.raises(ValueError, match="page_size"):
        fat.kv_block_scores(q, bounds, table, lens, more + 16)
    with pytest.raises(ValueError, match="num_blocks"):
        fat.attn_decode_sparse(q, cache.k, cache.v, table, lens, scores, more + 2)
    with pytest.raises(ValueError, match="max_len"):
        fat.kv_cache_read(cache.k, cache.v, table, lens, more + 40)
    with pytest.raises(ValueError, match="new_tokens"):
        fat.kv_block_bounds(cache.k, table, lens, bounds, more + 1)
    token = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="tokens"):
        fat.kv_cache_write(token.expand(more + 1, 2, 64), token.expand(more + 1, 2, 64), cache.k,
                           cache.v, torch.zeros(1, dtype=torch.int64, device="cuda").expand(more + 1))
