"""Attention of drafted tokens whose waits inside the kernel run out: the call ends, the status says
so, nothing is left behind, and the next call is right."""
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from drafted_helpers import as_tensor, random_trees
from paged_helpers import TYPES, Cache, make_table, pages_for

pytestmark = pytest.mark.gpu

CASES = [
    # lens, T, heads, group, page size, d, query type, cache type, positions more in the table
    ([200], 8, 2, 4, 16, 128, "bf16", "bf16", 0),
    ([2000, 300, 129], 8, 2, 4, 64, 128, "bf16", "bf16", 0),  # one block of rows
    ([2000, 300, 129], 64, 2, 4, 64, 128, "bf16", "bf16", 3400),  # two
    ([40 + 60 * i for i in range(40)], 5, 8, 2, 32, 64, "fp16", "fp16", 3400),
    ([1500, 128, 100, 90], 64, 2, 3, 16, 64, "fp16", "fp16", 3400),
    ([200], 8, 2, 4, 16, 128, "bf16", "e4m3", 0),
    ([2000, 300, 129], 8, 2, 4, 64, 128, "bf16", "e4m3", 3400),  # rows that stand twice
    ([30 + 40 * i for i in range(40)], 40, 8, 3, 32, 64, "fp16", "e4m3", 3400),
]
# many tiles and items to a thread block: some waits are longer than what the shortest limits allow,
# in any case (the producers' for room)
LONG = [
    ([40 + 60 * i for i in range(60)], 5, 8, 2, 32, 64, "fp16", "fp16", 3400),
    ([100 + 90 * i for i in range(60)], 64, 8, 4, 64, 128, "bf16", "bf16", 0),
    ([100 + 90 * i for i in range(60)], 64, 8, 3, 16, 64, "fp16", "fp16", 0),
    ([100 + 90 * i for i in range(60)], 8, 8, 4, 64, 128, "bf16", "e4m3", 0),
    ([100 + 90 * i for i in range(60)], 40, 8, 3, 32, 64, "fp16", "e4m3", 0),
]


def arguments(case):
    lens, T, heads, group, page_size, d, q_type, kind, more = case
    cache = Cache(pages_for(lens, page_size), heads, page_size, d, kind, seed=3)
    width = max(-(-n // page_size) for n in lens) + -(-more // page_size)
    table = make_table(lens, page_size, cache.k.shape[0], seed=3, width=width)
    g = torch.Generator().manual_seed(4)
    q = torch.randn((len(lens), T, heads * group, d), generator=g).to(TYPES[q_type])
    args = (q.cuda(), cache.k, cache.v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            as_tensor(random_trees(len(lens), T, 5)).cuda())
    drafted = torch.tensor([min(n, T) for n in lens], dtype=torch.int32).cuda()
    return args, dict(cache.scale_args, draft_lens=drafted)


@pytest.mark.parametrize("case", CASES + LONG, ids=lambda c: "-".join(map(str, c[1:])))
def test_a_wait_that_runs_out(cuda_device, case):
    args, kw = arguments(case)
    want = fat.attn_tree_paged(*args, **kw)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    for limit in (1, 100, 500, 1000, 2000, 3000, 5000, 8000, 12000, 20000):
        fat.attn_tree_paged(*args, **kw, wait_timeout_ns=limit)
        status = fat.check_device_error()
        # (whether a wait takes longer than its limit is the machine's, but for these)
        assert status == fat.FAT_ERR_DEVICE_TIMEOUT if case in LONG and limit <= 100 else \
            status in (fat.FAT_OK, fat.FAT_ERR_DEVICE_TIMEOUT), limit
        got = fat.attn_tree_paged(*args, **kw)
        torch.cuda.synchronize()
        assert fat.check_device_error() == fat.FAT_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want)), limit


def test_a_limit_that_is_long_enough(cuda_device):
    args, kw = arguments(CASES[1])
    want = fat.attn_tree_paged(*args, **kw)
    got = fat.attn_tree_paged(*args, **kw, wait_timeout_ns=2 * 10 ** 9)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (-1, 1 << 63):
        with pytest.raises(ValueError, match="wait_timeout_ns"):
            fat.attn_tree_paged(*args, **kw, wait_timeout_ns=bad)
