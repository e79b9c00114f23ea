"""Calls of the paged operators with a stream of their own: what they allocate is neither in use
on the current stream any more, nor given away while the current stream still reads it."""
import pytest
import torch

import tensorized_online_softmax_gb300 as fat
from paged_helpers import Cache, make_table, pages_for, queries

pytestmark = pytest.mark.gpu

LENS, HEADS, GROUP, PAGE, D = [5000, 700, 40], 2, 4, 64, 128
WAIT = 40_000_000  # cycles: some 20 ms, far above a call's host and device time


def calls():
    """name -> (call with a stream or None, the shapes and types that it allocates)."""
    cache = Cache(pages_for(LENS, PAGE), HEADS, PAGE, D, "e4m3", seed=1)
    table = make_table(LENS, PAGE, cache.k.shape[0], seed=1).cuda()
    lens = torch.tensor(LENS, dtype=torch.int32).cuda()
    q = queries(3, HEADS * GROUP, D, "bf16", seed=1).cuda()
    bounds = torch.randn((cache.k.shape[0], HEADS, 2, D), device="cuda").to(torch.bfloat16)
    scores = torch.randn((3, HEADS, table.shape[1]), device="cuda")
    kw = cache.scale_args
    return {
        "read": lambda s: fat.kv_cache_read(cache.k, cache.v, table, lens, 5000, stream=s, **kw),
        "decode": lambda s: fat.attn_decode_paged(q, cache.k, cache.v, table, lens, stream=s, **kw),
        "scores": lambda s: (fat.kv_block_scores(q, bounds, table, lens, PAGE, stream=s),),
        "sparse": lambda s: fat.attn_decode_sparse(q, cache.k, cache.v, table, lens, scores, 20,
                                                   stream=s, **kw),
    }


def overwrite(tensors):
    """New tensors like those and like a workspace, filled, and let go of."""
    work = fat.attn_decode_workspace_bytes(3, HEADS * GROUP, HEADS, D, 20)
    new = [torch.empty_like(t) for t in tensors]
    for t in new + [torch.empty(work, dtype=torch.uint8, device="cuda")]:
        t.view(torch.uint8).fill_(0xFF)


@pytest.mark.parametrize("name", ["read", "decode", "scores", "sparse"])
@pytest.mark.parametrize("as_number", [False, True], ids=["stream", "handle"])
def test_outputs_are_not_memory_that_the_current_stream_still_writes(cuda_device, name, as_number):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    given = side.cuda_stream if as_number else side
    for _ in range(2):  # (loads what is to be loaded; memory or kernels that are new would wait)
        call(given)
        overwrite(want)
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(WAIT)
        overwrite(want)  # (after the wait, but the memory is free for the next allocation now)
        got = call(given)
        side.synchronize()
        early = torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        assert not early, "the current stream was done too soon to show anything"
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got


@pytest.mark.parametrize("name", ["read", "decode", "scores", "sparse"])
def test_outputs_let_go_of_while_the_current_stream_reads_them(cuda_device, name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    [t.clone() for t in call(side)]
    overwrite(want + want)
    with torch.cuda.stream(side):
        overwrite(want + want)
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(WAIT)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):  # the next owners of that memory, if it were free
        overwrite(want + want)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


def test_a_workspace_is_free_for_its_own_stream_only(cuda_device):
    """The workspace of a call is let go of on return, with its kernels still to run."""
    call = calls()["decode"]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    [t.clone() for t in call(side)]
    overwrite(want + want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(side)
    overwrite(want + want)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["read", "decode", "scores", "sparse"])
def test_a_side_stream_inside_a_captured_graph(cuda_device, name):
    """The given stream forks from the capturing one and joins it again."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        first = call(side)
        second = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in first + second:
            t.view(torch.uint8).fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for got in (first, second) for a, b in zip(got, want))


def test_the_default_stream_by_its_number(cuda_device):
    call = calls()["decode"]
    want = call(None)
    got = call(0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
