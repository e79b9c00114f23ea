"""Drafted tokens over the paged cache where magnitudes lie far apart, caches are large or
broadcast, and calls meet: on several threads, on other streams, in one captured graph."""
import math
import threading

import numpy as np
import pytest
import torch

import drafted_reference
import tensorized_online_softmax_gb300 as fat
from drafted_helpers import WEIGHT, angle_table, as_tensor, check_tree, random_trees
from paged_helpers import TYPES, Cache, make_table, pages_for, ref

pytestmark = pytest.mark.gpu


WIDE = False


@pytest.fixture(params=[False, True], ids=["table", "long_table"], autouse=True)
def table_length(request):
    """A table for the sequences, whose items are mostly not split, and one for 3400 positions more,
    where they are."""
    global WIDE
    WIDE = request.param


class Drafted:
    """Sequences whose keys and values [tokens, heads, d] kv_cache_write has stored."""

    def __init__(self, lens, T, q, k, v, kind, page_size=16, seed=0, scales=None):
        self.lens, self.T, self.q = lens, T, q
        heads, d = k.shape[1:]
        self.cache = Cache(pages_for(lens, page_size), heads, page_size, d, kind, seed=seed)
        width = max(-(-n // page_size) for n in lens) + (-(-3400 // page_size) if WIDE else 0)
        self.table = make_table(lens, page_size, self.cache.k.shape[0], seed=seed, width=width)
        slots = torch.cat([self.table[b, torch.arange(n) // page_size].long() * page_size
                           + torch.arange(n) % page_size for b, n in enumerate(lens)])
        fat.kv_cache_write(k.cuda(), v.cuda(), self.cache.k, self.cache.v, slots.cuda(),
                           **self.cache.scale_args)
        self.masks = random_trees(len(lens), T, seed)
        self.scale = float(np.float32(d ** -0.5))

    def run(self, **kw):
        got = fat.attn_tree_paged(self.q.cuda(), self.cache.k, self.cache.v, self.table.cuda(),
                                  torch.tensor(self.lens, dtype=torch.int32).cuda(),
                                  as_tensor(self.masks).cuda(), **self.cache.scale_args, **kw)
        torch.cuda.synchronize()
        assert fat.check_device_error() == fat.FAT_OK
        return got

    def want(self, scale=None):
        return drafted_reference.tree(self.q.double(), *self.cache.held(), self.table, self.lens,
                                      [self.T] * len(self.lens), self.masks,
                                      self.cache.page_size, scale or self.scale)

    def positions(self, b, t):
        """Those that token t of sequence b sees, as pages and places."""
        context = self.lens[b] - self.T
        at = [j for j in range(self.lens[b])
              if drafted_reference.sees(j, context, self.masks[b][t], 0, 0)]
        ps = self.cache.page_size
        return torch.tensor([int(self.table[b, j // ps]) for j in at]), \
            torch.tensor([j % ps for j in at])


def sinks(lens, T, heads, group, d, typ, gap, seed):
    """Queries near one direction of signs for each head, keys whose scores are near 0 but for two
    positions of each sequence's context, which are `gap` above; values around a mean."""
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    u = torch.sign(torch.randn((heads, d), generator=g))
    q = u[:, None] + 0.2 * torch.randn((len(lens), T, heads, group, d), generator=g)
    k = 0.2 * torch.randn((n, heads, d), generator=g)
    v = 0.3 + 0.2 * torch.randn((n, heads, d), generator=g)
    at, start = [], 0
    for m in lens:
        at += [start + m // 3, start + m - 1 - T]
        start += m
    k[at] = u * (gap / math.sqrt(d))  # scale = 1 / sqrt(d): u . k / sqrt(d) = gap
    return q.reshape(len(lens), T, heads * group, d).to(TYPES[typ]), k, v, at


@pytest.mark.parametrize("kind,typ", [("fp16", "fp16"), ("bf16", "bf16"), ("e4m3", "fp16"),
                                      ("e4m3", "bf16")])
@pytest.mark.parametrize("lens,T,group", [([200, 41], 3, 4), ([2500], 40, 4)], ids=str)
@pytest.mark.parametrize("gap", [14.0, 16.1, 18.5, 20.3])
def test_weights_far_below_the_largest(cuda_device, kind, typ, lens, T, group, gap):
    """One key's score is `gap` above all others, which are equal, and its value is zero in all
    columns but one: the others alone make up the rest.  fp16 weights are off by at most 2^-25
    where the largest is at least 2^11: 2^-36 of it, times the sum of the values' magnitudes."""
    d = 64
    q, k, v, at = sinks(lens, T, 1, group, d, typ, gap, seed=21)
    top = k[at].clone()
    k.zero_()
    k[at] = top
    v[at] = 0
    v[at, :, 7] = 1.0
    v = v * (1.0 if kind == "bf16" else 64.0)
    s = Drafted(lens, T, q, k.to(TYPES[typ]), v.to(TYPES[typ]), kind, seed=9)
    want = s.want()
    if kind != "bf16":
        kk, vv = s.cache.held()
        for b in range(len(lens)):
            for t in range(T):
                at = s.positions(b, t)
                values = vv[at[0], 0, at[1]].abs().sum(0)
                for h in range(group):
                    p = torch.softmax(kk[at[0], 0, at[1]] @ q[b, t, h].double() * s.scale, 0)
                    want[2][b, t, h] += 2.0 ** -36 * p.max() * values / WEIGHT[q.dtype]
    check_tree(*s.run(), *want, what=f"{kind} {gap}")


@pytest.mark.parametrize("typ", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,T,group", [([300], 3, 4), ([2000], 40, 4)], ids=str)
def test_infinite_values_of_little_weight(cuda_device, typ, lens, T, group):
    """An infinite value makes its column infinite, 20 nats (2^-29 of the largest weight) below the
    largest score as well."""
    d = 64
    q, k, v, at = sinks(lens, T, 1, group, d, typ, 1.0, seed=31)
    u = torch.sign(k[at[0], 0])
    k = k * 0.02
    k[at[0]] = u * (20.0 / math.sqrt(d))
    low = [5, 110, 111, 250, lens[0] - T - 2]
    for i, (j, gap) in enumerate(zip(low, (0.0, 4.0, 8.0, 12.0, 17.0))):
        k[j] = u * (gap / math.sqrt(d))
        v[j, 0, 2 * i] = math.inf
        v[j, 0, 2 * i + 1] = -math.inf
    s = Drafted(lens, T, q, k.to(TYPES[typ]), v.to(TYPES[typ]), typ, seed=9)
    o, lse = s.run()
    want = s.want()
    check_tree(o, lse, want[0], want[1],
               torch.where(torch.isfinite(want[2]), want[2], torch.zeros_like(want[2])))
    assert torch.isinf(o[..., :10]).all() and torch.isfinite(o[..., 10:]).all()


@pytest.mark.parametrize("kind,typ", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"),
                                      ("e4m3", "fp16")])
@pytest.mark.parametrize("T,group", [(5, 2), (40, 4)])
def test_queries_that_are_not_finite(cuda_device, kind, typ, T, group):
    """NaN for their own rows, nothing for the others."""
    g = torch.Generator().manual_seed(33)
    lens = [T + 200, T + 40]
    q = torch.randn((2, T, group, 64), generator=g).to(TYPES[typ])
    k, v = torch.randn((2, sum(lens), 1, 64), generator=g).to(TYPES[typ])
    q[0, 1, 0, 7], q[1, 2, 1, 60], q[1, 0, 0] = math.nan, math.inf, -math.inf
    s = Drafted(lens, T, q, k, v, kind, seed=5)
    o, lse = s.run()
    bad = ~torch.isfinite(q).all(-1)
    assert torch.isnan(o[bad]).all() and not torch.isfinite(lse[bad]).any()
    check_tree(o[~bad], lse[~bad], *(x[~bad] for x in s.want()))


def test_more_sequences_than_threads(cuda_device):
    """The plan walks several sequences to a thread."""
    for kind, d in (("bf16", 64), ("e4m3", 128)):
        g = torch.Generator().manual_seed(34)
        lens = [2 + i % 5 + (300 if i % 97 == 0 else 0) for i in range(2000)]
        q = torch.randn((len(lens), 2, 2, d), generator=g).bfloat16()
        k, v = torch.randn((2, sum(lens), 1, d), generator=g).bfloat16()
        s = Drafted(lens, 2, q, k, v, kind, seed=5)
        check_tree(*s.run(), *s.want())


@pytest.mark.parametrize("typ", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,T,group", [([300, 40], 3, 4), ([2000, 50], 40, 4)], ids=str)
def test_infinite_keys(cuda_device, typ, lens, T, group):
    """A score of +inf has no softmax: NaN, for the rows whose query is positive there; a score of
    -inf has no weight.  The other sequence is as it was."""
    q, k, v, _ = sinks(lens, T, 1, group, 64, typ, 2.0, seed=32)
    q[0, :, :, 3] = torch.tensor([1.0, -1.0, 0.5, -0.25])
    k[77, 0, 3] = math.inf
    s = Drafted(lens, T, q, k.to(TYPES[typ]), v.to(TYPES[typ]), typ, seed=9)
    o, lse = s.run()
    want = s.want()
    assert torch.isnan(want[0][0, :, ::2]).all() and torch.isfinite(want[0][0, :, 1::2]).all()
    assert torch.isnan(o[0, :, ::2]).all() and not torch.isfinite(lse[0, :, ::2]).any()
    check_tree(o[0, :, 1::2], lse[0, :, 1::2], *(x[0, :, 1::2] for x in want))
    check_tree(o[1], lse[1], *(x[1] for x in want))


@pytest.mark.parametrize("T,group", [(4, 2), (40, 3)])
def test_queries_of_a_wide_range(cuda_device, T, group):
    """bf16 queries over an e4m3 cache: sequences whose queries are powers of two away from the
    others', against keys that are as many away the other way, and rows (and elements) of unlike
    magnitude side by side."""
    d, g = 64, torch.Generator().manual_seed(41)
    powers = [0, 40, -40, 90, -90, 118, -118]
    lens = [T + 150] * (len(powers) + 2)
    q = torch.randn((len(lens), T, group, d), generator=g)
    k = torch.randn((sum(lens), 1, d), generator=g)
    v = torch.randn((sum(lens), 1, d), generator=g)
    for b, n in enumerate(powers):
        q[b] *= 2.0 ** n
        k[b * lens[0]:(b + 1) * lens[0]] *= 2.0 ** -n
    b = len(powers)
    q[b, ::2] *= 2.0 ** -60  # (rows that score next to nothing)
    q[b + 1, :, :, ::2] *= 2.0 ** -50  # within a row
    s = Drafted(lens, T, q.bfloat16(), k.bfloat16(), v.bfloat16(), "e4m3", seed=7)
    check_tree(*s.run(), *s.want())


@pytest.mark.parametrize("q_type", ["bf16", "fp16"])
@pytest.mark.parametrize("T,group,d", [(4, 2, 128), (40, 3, 64), (5, 3, 64)])
def test_scales_that_fp16_has_not(cuda_device, q_type, T, group, d):
    """Rows of an e4m3 cache whose scales, or whose values, are not fp16's: in some tiles keys, in
    some values, in some both; zero rows; the rows not seen hold any scale."""
    lens = [T + 700, T + 130, T]
    g = torch.Generator().manual_seed(51)
    n = sum(lens)
    q = torch.randn((len(lens), T, group, d), generator=g).to(TYPES[q_type])
    k = torch.randn((n, 1, d), generator=g)
    v = torch.randn((n, 1, d), generator=g)
    k[100:140] *= 2.0 ** -30
    k[300:301] *= 2.0 ** -100
    k[500:520] = 0
    big = 30 if q_type == "bf16" else 15  # (the results are of the queries' type)
    v[200:230] *= 2.0 ** big
    v[400:401] *= 2.0 ** -40
    v[520:640] *= 2.0 ** min(big, 20)
    v[700:710] = 0
    s = Drafted(lens, T, q, k.bfloat16(), v.bfloat16(), "e4m3", seed=8)
    # keys of small codes and large scales: 2^-9 2^(135 - 127) and so on
    for j in (10, 130, 600):
        at = int(s.table[0, j // 16]), 0, j % 16
        s.cache.k.view(torch.uint8)[at] = torch.randint(0, 4, (d,), generator=g,
                                                        dtype=torch.uint8).cuda()
        s.cache.scales[0][at] = 135
    free = set(range(s.cache.k.shape[0])) - {int(x) for x in s.table.flatten()}
    for page in free:
        for x in s.cache.scales:
            x[page] = torch.arange(16, dtype=torch.uint8, device="cuda") * 16 + 14
    last = int(s.table[0, (lens[0] - 1) // 16])
    for x in s.cache.scales:
        x[last, 0, lens[0] % 16 or 16:] = 250
    check_tree(*s.run(), *s.want())


@pytest.mark.parametrize("q_type", ["bf16", "fp16"])
@pytest.mark.parametrize("T,group,d", [(4, 2, 128), (40, 3, 64)])
def test_many_items_with_and_without_such_scales(cuda_device, q_type, T, group, d):
    """Blocks that go from one sequence's head to the next, whose tiles' keys and values have
    scales that fp16 has, or has not, at random: what a tile is must not be told from another's."""
    g = torch.Generator().manual_seed(71)
    lens = [T + 130 * (1 + i % 9) for i in range(60)]
    n = sum(lens)
    q = torch.randn((len(lens), T, 3 * group, d), generator=g).to(TYPES[q_type])
    k = torch.randn((n, 3, d), generator=g)
    v = torch.randn((n, 3, d), generator=g)
    at = 0
    for m in lens:
        for j in range(0, m, 128):
            w = slice(at + j, at + min(j + 128, m))
            for h in range(3):
                if torch.rand((), generator=g) < 0.4:
                    k[w, h] *= 2.0 ** -24
                if torch.rand((), generator=g) < 0.4:
                    v[w, h] *= 2.0 ** -24
        at += m
    s = Drafted(lens, T, q, k.bfloat16(), v.bfloat16(), "e4m3", page_size=64, seed=12)
    kk, vv = s.cache.held()
    for turn in range(3):
        o, lse = s.run()
        for b in range(turn, len(lens), 3):
            for t in (0, T - 1):
                at = s.positions(b, t)
                for h in range(3):
                    r = slice(h * group, (h + 1) * group)
                    want = ref.attend(s.q[b, t, r].double(), kk[at[0], h, at[1]],
                                      vv[at[0], h, at[1]], s.scale)
                    check_tree(o[b, t, r], lse[b, t, r], *want, what=f"{b} {t} {h}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,group", [(1, 129), (3, 200), (2, 300)])
def test_many_query_heads_to_a_cached_one(cuda_device, kind, T, group):
    g = torch.Generator().manual_seed(61)
    lens = [T + 140, T]
    q = torch.randn((2, T, group, 64), generator=g).bfloat16()
    k, v = torch.randn((2, sum(lens), 1, 64), generator=g).bfloat16()
    s = Drafted(lens, T, q, k, v, kind, seed=6)
    check_tree(*s.run(), *s.want())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_broadcast_views(cuda_device, kind):
    """One head's rows for all heads, one page for all pages, one sequence's queries for all: the
    same bits as of tensors of their own."""
    g = torch.Generator().manual_seed(62)
    cache = Cache(6, 1, 16, 128, kind, seed=3)
    q = torch.randn((1, 5, 8, 128), generator=g).bfloat16().cuda()
    table = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32).cuda()
    lens = torch.tensor([40, 21], dtype=torch.int32).cuda()
    tree = as_tensor(random_trees(2, 5)).cuda()
    for turn in ("heads", "pages"):
        def view(x):
            tail = (-1,) * (x.dim() - 2)
            return x.expand(6, 4, *tail) if turn == "heads" else x[:1].expand(6, 1, *tail)
        k, v = view(cache.k), view(cache.v)
        own = [x.contiguous() for x in (k, v)]
        scales = {n: None if x is None else view(x).contiguous()
                  for n, x in cache.scale_args.items()}
        wide = q.expand(2, -1, -1, -1)
        got = fat.attn_tree_paged(wide, k, v, table, lens, tree, **scales)
        want = fat.attn_tree_paged(wide.contiguous(), *own, table, lens, tree, **scales)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = fat.attn_decode_window(wide[:, 0], k, v, table, lens, 17, 2, **scales)
        want = fat.attn_decode_window(wide[:, 0].contiguous(), *own, table, lens, 17, 2, **scales)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # heads or tokens that share memory are refused, not copied without a word
        for shared in (q[:, :, :1].expand(2, 5, 8, 128), q[:, :1].expand(2, 5, 8, 128)):
            with pytest.raises(fat.FatError, match="UNSUPPORTED"):
                fat.attn_tree_paged(shared, k, v, table, lens, tree, **scales)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK


def test_offsets_past_32_bits(cuda_device):
    """A cache of 5 GiB a side: the last pages are written, moved and attended to in place."""
    pages, H, ps, d, T, G = 42000, 8, 64, 128, 6, 2
    k = torch.empty((pages, H, ps, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() * 2 > 2 ** 32
    n = 100
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32)
    at = torch.arange(n)
    slots = table[0].long()[at // ps] * ps + at % ps
    g = torch.Generator().manual_seed(1)
    x = torch.randn((2, n, H, d), generator=g).bfloat16()
    still = torch.cat([torch.ones(1, d // 2), torch.zeros(1, d // 2)], 1).cuda()  # no rotation
    dev = [t.cuda() for t in (x[0], x[1], slots)]
    fat.kv_cache_append(None, *dev[:2], k, v, dev[2], torch.zeros(n, dtype=torch.int64).cuda(),
                        still)
    q = torch.randn((1, T, H * G, d), generator=g).bfloat16()
    masks = random_trees(1, T, 1)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    own_k, own_v = (t.transpose(1, 2).reshape(-1, H, ps, d).double() for t in
                    torch.cat([x, torch.zeros((2, 128 - n, H, d))], 1).reshape(2, 2, ps, H, d))
    near = torch.tensor([[0, 1]])
    got = fat.attn_tree_paged(q.cuda(), k, v, table.cuda(), lens, as_tensor(masks).cuda())
    scale = float(np.float32(d ** -0.5))
    check_tree(*got, *drafted_reference.tree(q.double(), own_k, own_v, near, [n], [T], masks, ps,
                                             scale))
    path = [1, 4]
    fat.kv_cache_keep(k, v, table.cuda(), lens - T, torch.tensor([path], dtype=torch.int32).cuda(),
                      torch.tensor([2], dtype=torch.int32).cuda())
    for t in (own_k, own_v):
        drafted_reference.keep(t, near, [n - T], [path], [2], ps)
    now = n - T + 2
    o, lse = fat.attn_decode_window(q[:, 0].cuda(), k, v, table.cuda(), lens - T + 2, 50, 3)
    check_tree(o, lse, *drafted_reference.window(q[:, 0].double(), own_k, own_v, near, [now], ps,
                                                 scale, 50, 3))
    assert fat.check_device_error() == fat.FAT_OK
    del k, v
    torch.cuda.empty_cache()


class Step:
    """A step of drafted tokens of one batch: stored, judged, the accepted ones kept, and a single
    token's windowed attention."""

    def __init__(self, kind, d, seed, T=6, H=2, G=3, ps=16):
        g = torch.Generator().manual_seed(seed)
        self.context = [40 + 17 * seed, 3, 200]
        B, room = 3, [n + T + 2 for n in self.context]
        self.cache = Cache(pages_for(room, ps), H, ps, d, kind, seed=seed)
        self.first = [x.clone() for x in self.tensors()]
        width = max(-(-n // ps) for n in room) + (-(-3400 // ps) if WIDE else 0)
        table = make_table(room, ps, self.cache.k.shape[0], seed=seed, width=width)
        slots = [int(table[b, j // ps]) * ps + j % ps for b, n in enumerate(self.context)
                 for j in range(n, n + T)]
        dev = lambda x, t=None: torch.as_tensor(x, dtype=t).cuda()
        rows = [torch.randn((B * T, h, d), generator=g).bfloat16().cuda() for h in (H * G, H, H)]
        self.append_args = (*rows, self.cache.k, self.cache.v, dev(slots),
                            dev([n + i for n in self.context for i in range(T)]),
                            angle_table(300, d).cuda())
        self.shape = B, T, H * G, d
        self.table, self.lens = dev(table), dev(self.context, torch.int32)
        self.tree = as_tensor(random_trees(B, T, seed)).cuda()
        self.path = dev([[0, 3], [2, 5], [0, 1]], torch.int32)
        self.counts = dev([2, 1, 0], torch.int32)

    def tensors(self):
        return [x.view(torch.uint8) for x in (self.cache.k, self.cache.v, *self.cache.scales)
                if x is not None]

    def reset(self):
        for x, y in zip(self.tensors(), self.first):
            x.copy_(y)

    def run(self, stream=None):
        kw = dict(self.cache.scale_args, stream=stream)
        c = self.cache
        q = fat.kv_cache_append(*self.append_args, **kw)
        # (plain operations on the current stream would not be ordered with `stream`)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            lens, kept = self.lens + self.shape[1], self.lens + self.counts
        out = fat.attn_tree_paged(q.view(self.shape), c.k, c.v, self.table, lens, self.tree, **kw)
        fat.kv_cache_keep(c.k, c.v, self.table, self.lens, self.path, self.counts, **kw)
        one = fat.attn_decode_window(q.view(self.shape)[:, 0], c.k, c.v, self.table, kept, 30, 2,
                                     **kw)
        return [q, *out, *one]


def test_a_step_in_one_graph(cuda_device):
    """All four calls in one captured graph; replayed with new lengths, trees and paths."""
    for kind in ("bf16", "e4m3"):
        s = Step(kind, 128, 1)
        s.run()
        s.reset()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.run()
        for turn in range(2):
            s.reset()
            graph.replay()
            torch.cuda.synchronize()
            got = [x.clone() for x in out + s.tensors()]
            s.reset()
            want = s.run() + s.tensors()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (kind, turn)
            s.tree.copy_(as_tensor(random_trees(3, 6, 99)))
            s.path.copy_(torch.tensor([[1, 4], [0, 0], [0, 5]]))
            s.counts.copy_(torch.tensor([2, 0, 2]))
    assert fat.check_device_error() == fat.FAT_OK


def test_a_step_on_another_stream(cuda_device):
    """With stream= all of it runs there, outputs included: the current stream is busy."""
    s = Step("e4m3", 64, 2)
    want = [x.clone() for x in s.run() + s.tensors()]
    s.reset()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = s.run(stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + s.tensors(), want))
    assert fat.check_device_error() == fat.FAT_OK


def test_steps_on_several_threads(cuda_device):
    """Host threads with a stream each, whole steps over caches of their own."""
    steps = [Step(("bf16", "e4m3")[i % 2], (64, 128)[i // 2], 3 + i) for i in range(4)]
    want = []
    for s in steps:
        want.append([x.clone() for x in s.run() + s.tensors()])
        s.reset()
    torch.cuda.synchronize()
    got, errors = [[] for _ in steps], []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    steps[i].reset()
                    got[i].append([x.clone() for x in steps[i].run() + steps[i].tensors()])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # told by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for w, g in zip(want, got):
        assert len(g) == 8 and all(torch.equal(a, b) for x in g for a, b in zip(x, w))
    assert fat.check_device_error() == fat.FAT_OK


def test_what_requires_a_gradient_is_refused(cuda_device):
    s = Step("bf16", 64, 1)
    for i in (0, 1, 2, 3, 4, 7):
        args = list(s.append_args)
        args[i] = args[i].clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            fat.kv_cache_append(*args)
        with torch.no_grad():
            fat.kv_cache_append(*args)
    with torch.inference_mode():
        s.run()
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
