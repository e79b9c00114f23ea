"""The paged operators have no backward pass: what requires a gradient is refused, not cut off."""
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import Cache, make_table, pages_for, queries

pytestmark = pytest.mark.gpu


def calls():
    """name -> (call, its arguments that could require a gradient)."""
    lens = [40, 7]
    cache = Cache(pages_for(lens, 16), 2, 16, 64, "bf16", seed=1)
    table = make_table(lens, 16, cache.k.shape[0]).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    q = queries(2, 4, 64, "bf16").cuda()
    new = torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([3, 40], device="cuda")
    bounds = torch.zeros((cache.k.shape[0], 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros((2, 2, table.shape[1]), device="cuda")
    kv = dict(k_cache=cache.k, v_cache=cache.v)
    at = dict(page_table=table, seq_lens=n)
    return {
        "write": (lambda **a: fat.kv_cache_write(slots=slots, **a), dict(k=new, v=new.clone(), **kv)),
        "read": (lambda **a: fat.kv_cache_read(max_len=40, **at, **a), kv),
        "decode": (lambda **a: fat.attn_decode_paged(**at, **a), dict(q=q, **kv)),
        "bounds": (lambda **a: fat.kv_block_bounds(**at, **a),
                   dict(k_cache=cache.k, bounds=bounds)),
        "scores": (lambda **a: fat.kv_block_scores(page_size=16, **at, **a),
                   dict(q=q, bounds=bounds)),
        "sparse": (lambda **a: fat.attn_decode_sparse(num_blocks=2, **at, **a),
                   dict(q=q, scores=scores, **kv)),
    }


@pytest.mark.parametrize("name", ["write", "read", "decode", "bounds", "scores", "sparse"])
def test_what_requires_a_gradient_is_refused(cuda_device, name):
    call, args = calls()[name]
    call(**args)
    for which in args:
        asks = {**args, which: args[which].clone().requires_grad_()}
        with pytest.raises(ValueError, match="gradient"):
            call(**asks)
        with torch.no_grad():
            call(**asks)
        with torch.inference_mode():
            call(**asks)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
