"""Single-token attention over a sliding window with sinks, against the plain 64-bit
implementation."""
import math

import numpy as np
import pytest
import torch

import drafted_reference
import tensorized_online_softmax_gb300 as fat
from paged_helpers import BEHIND, Cache, check_attention, make_table, pages_for, queries

pytestmark = pytest.mark.gpu


def setup(lens, heads, group, page_size, d, q_type, kind, layout="phtd", seed=0, width=None):
    cache = Cache(pages_for(lens, page_size), heads, page_size, d, kind, layout, seed=seed)
    if width is None:
        width = max(1, max(-(-n // page_size) for n in lens)) + 2
    table = make_table(lens, page_size, cache.k.shape[0], seed=seed, width=width)
    return cache, table, lens, queries(len(lens), heads * group, d, q_type, seed=seed)


def given_back(table, lens, page_size, window, sinks):
    """The table with the entries of pages that nobody sees out of range."""
    table = table.clone()
    for b, n in enumerate(lens):
        for i in range(-(-n // page_size)):
            if not any(j < sinks or j >= n - window
                       for j in range(i * page_size, min(n, (i + 1) * page_size))):
                table[b, i] = BEHIND
    return table


def run(cache, table, lens, q, window, sinks, **kw):
    o, lse = fat.attn_decode_window(q.cuda(), cache.k, cache.v, table.cuda(),
                                    torch.tensor(lens, dtype=torch.int32).cuda(), window, sinks,
                                    **cache.scale_args, **kw)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    return o, lse


def check(cache, table, lens, q, window, sinks, what=""):
    scale = float(np.float32(q.shape[-1] ** -0.5))
    o, lse = run(cache, given_back(table, lens, cache.page_size, window, sinks), lens, q, window,
                 sinks)
    want = drafted_reference.window(q.double(), cache.k_values, cache.v_values, table, lens,
                                    cache.page_size, scale, window, sinks)
    check_attention(o, lse, *want, what=what, kind=cache.kind)
    return o, lse


CASES = [
    # lens, heads, group, page_size, d, query type, cache type, layout
    ([0, 1, 2, 40, 100, 129], 2, 1, 16, 128, "bf16", "bf16", "phtd"),
    ([700, 63, 511, 1000], 2, 4, 64, 128, "bf16", "bf16", "pthd"),
    ([900, 0, 65, 700], 1, 8, 16, 128, "bf16", "e4m3", "phtd"),
    ([800, 33], 2, 3, 32, 64, "fp16", "e4m3", "kv"),
    ([1000, 64, 640], 1, 16, 128, 64, "fp16", "fp16", "kv"),
    ([900, 20], 1, 20, 256, 64, "bf16", "bf16", "phtd"),
]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (64, 64), (100, 0), (128, 70),
                                          (333, 200), (2000, 3), (600, 2000)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
def test_window(cuda_device, case, window, sinks):
    lens, *rest = case
    check(*setup(lens, *rest, seed=len(lens)), window, sinks, f"{case} {window} {sinks}")


def test_a_window_as_long_as_the_sequences_is_decode(cuda_device):
    cache, table, lens, q = setup([700, 1, 0, 333, 512], 2, 4, 16, 128, "bf16", "bf16", seed=3)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    want = fat.attn_decode_paged(q.cuda(), cache.k, cache.v, table.cuda(), n)
    for window, sinks in ((700, 0), (2 ** 31 - 1, 2 ** 31 - 1), (350, 350), (1, 10 ** 6)):
        got = run(cache, table, lens, q, window, sinks)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
def test_what_is_not_seen_has_no_part(cuda_device, kind):
    """NaN and infinities in the gap, in the rest of the pages at its borders and behind."""
    window, sinks = 77, 21
    cache, table, lens, q = setup([500, 130, 97, 99, 0], 2, 2, 16, 128,
                                  "fp16" if kind == "fp16" else "bf16", kind, seed=4)
    want = check(cache, table, lens, q, window, sinks)
    seen = torch.zeros(cache.k.shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            if j < sinks or j >= n - window:
                seen[table[b, j // 16], j % 16] = True
    hidden = ~seen[:, None, :, None].cuda().expand(cache.k.shape)
    for fill in (math.nan, math.inf):
        for t in (cache.k, cache.v):
            if kind == "e4m3":
                t.view(torch.uint8)[hidden] = 0x7F
            else:
                t[hidden] = fill
        if kind == "e4m3":
            for s in cache.scales:
                s[hidden[..., 0]] = 255
        got = run(cache, table, lens, q, window, sinks)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_long_sequences_split_over_the_blocks(cuda_device):
    """Windows long enough that every thread block gets part of one; the pages at once, as the
    loop of the reference is slow here."""
    for lens, window, sinks in (([50000], 30000, 100), ([20000, 0, 9000, 40000, 5], 7001, 65)):
        cache, table, lens, q = setup(lens, 1, 2, 64, 64, "bf16", "bf16", seed=5)
        o, lse = run(cache, given_back(table, lens, 64, window, sinks), lens, q, window, sinks)
        for b, n in enumerate(lens):
            ids = table[b, :-(-n // 64)].long()
            at = torch.arange(n)
            at = at[(at < sinks) | (at >= n - window)]
            k, v = (x[ids, 0].reshape(-1, 64)[at] for x in (cache.k_values, cache.v_values))
            want = drafted_reference.ref.attend(q[b].double(), k, v, 0.125)
            check_attention(o[b], lse[b], *want, what=f"{lens} {b}")


@pytest.mark.parametrize("batch,heads,group,kind,q_type", [
    (40, 4, 2, "bf16", "bf16"), (52, 8, 8, "e4m3", "bf16"), (160, 4, 1, "fp16", "fp16"),
    (30, 8, 16, "e4m3", "fp16"), (256, 4, 3, "bf16", "bf16")])
def test_many_short_windows(cuda_device, batch, heads, group, kind, q_type):
    """Enough items that each has a block of its own, in one wave of blocks or in several."""
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(0, 2200, batch)]
    lens[:5] = [0, 1, 800, 801, 2200]
    window, sinks = 800, 70
    cache, table, lens, q = setup(lens, heads, group, 64, 64, q_type, kind, seed=batch)
    o, lse = run(cache, given_back(table, lens, 64, window, sinks), lens, q, window, sinks)
    for b in [0, 1, 2, 3, 4, *range(5, batch, 9)]:
        n = lens[b]
        ids = table[b, :-(-n // 64)].long()
        at = torch.arange(n)
        at = at[(at < sinks) | (at >= n - window)]
        for h in range(heads):
            k, v = (x[ids, h].reshape(-1, 64)[at] for x in (cache.k_values, cache.v_values))
            r = slice(h * group, (h + 1) * group)
            if not n:
                assert (o[b, r] == 0).all() and (lse[b, r] == -math.inf).all()
                continue
            want = drafted_reference.ref.attend(q[b, r].double(), k, v, 0.125)
            check_attention(o[b, r], lse[b, r], *want, what=f"{b} {h}", kind=kind)


def test_graph_replays_with_new_lengths(cuda_device):
    cache, table, lens, q = setup([600, 40, 900], 2, 4, 16, 128, "bf16", "e4m3", seed=6)
    n = torch.tensor([100, 7, 5], dtype=torch.int32).cuda()
    args = q.cuda(), cache.k, cache.v, table.cuda(), n, 130, 20
    fat.attn_decode_window(*args, **cache.scale_args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fat.attn_decode_window(*args, **cache.scale_args)
    n.copy_(torch.tensor(lens, dtype=torch.int32))
    graph.replay()
    want = fat.attn_decode_window(*args, **cache.scale_args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_pages_and_lengths_are_reported(cuda_device):
    cache, table, lens, q = setup([300, 200], 2, 2, 16, 64, "bf16", "bf16", seed=7)
    for at, value in ((18, BEHIND), (18, -1), (0, 10 ** 6)):
        bad = table.clone()
        bad[0, at] = value
        o, _ = fat.attn_decode_window(q.cuda(), cache.k, cache.v, bad.cuda(),
                                      torch.tensor(lens, dtype=torch.int32).cuda(), 60, 3)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX
        good, _ = run(cache, table, lens, q, 60, 3)
        assert torch.equal(o[1], good[1])
    for n in (-1, 10 ** 6):
        fat.attn_decode_window(q.cuda(), cache.k, cache.v, table.cuda(),
                               torch.tensor([n, 200], dtype=torch.int32).cuda(), 60, 3)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX


def test_refusals(cuda_device):
    cache, table, lens, q = setup([1000, 200], 2, 2, 16, 64, "bf16", "bf16", seed=7)
    args = q.cuda(), cache.k, cache.v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for bad in ((0,), (-1,), (2 ** 31,), (5, -1), (5, 2 ** 31)):
        with pytest.raises(ValueError):
            fat.attn_decode_window(*args, *bad)
    with pytest.raises(ValueError, match="gradient"):
        fat.attn_decode_window(args[0].requires_grad_(), *args[1:], 5)
    with pytest.raises(fat.FatError, match="INVALID_ARG"):
        fat.attn_decode_window(q.cuda(), *args[1:], 500,
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
