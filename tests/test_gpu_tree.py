"""Attention of drafted tokens over the paged cache against the plain 64-bit implementation."""
import math

import numpy as np
import pytest
import torch

import drafted_reference
import tensorized_online_softmax_gb300 as fat
from drafted_helpers import as_tensor, check_tree, random_trees
from paged_helpers import BEHIND, TYPES, Cache, make_table, pages_for

pytestmark = pytest.mark.gpu


WIDE = False


@pytest.fixture(params=[False, True], ids=["table", "long_table"], autouse=True)
def table_length(request):
    """A table for a little more than the sequences, whose items are mostly not split, and one for
    3400 positions more, where they are."""
    global WIDE
    WIDE = request.param


class Setup:
    def __init__(self, lens, drafted, T, heads, group, page_size, d, q_type, kind, layout="phtd",
                 seed=0, masks=None, spread=0, width=None):
        self.lens, self.drafted, self.T = lens, drafted, T
        self.cache = Cache(pages_for(lens, page_size), heads, page_size, d, kind, layout,
                           seed=seed, spread=spread)
        if width is None:
            width = max(1, max(-(-n // page_size) for n in lens)) + 2
            if WIDE:
                width += -(-3400 // page_size)
        self.table = make_table(lens, page_size, self.cache.k.shape[0], seed=seed, width=width)
        g = torch.Generator().manual_seed(seed + 9)
        self.q = torch.randn((len(lens), T, heads * group, d), generator=g).to(TYPES[q_type])
        self.masks = masks or random_trees(len(lens), T, seed)
        self.scale = float(np.float32(d ** -0.5))

    def args(self, table=None):
        return (self.q.cuda(), self.cache.k, self.cache.v,
                (self.table if table is None else table).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda(), as_tensor(self.masks).cuda())

    def more(self, **kw):
        if any(n != self.T for n in self.drafted):
            kw["draft_lens"] = torch.tensor(self.drafted, dtype=torch.int32).cuda()
        return {**self.cache.scale_args, **kw}

    def run(self, table=None, **kw):
        o, lse = fat.attn_tree_paged(*self.args(table), **self.more(**kw))
        torch.cuda.synchronize()
        assert fat.check_device_error() == fat.FAT_OK
        return o, lse

    def want(self, window=None, sinks=0):
        return drafted_reference.tree(self.q.double(), self.cache.k_values, self.cache.v_values,
                                      self.table, self.lens, self.drafted, self.masks,
                                      self.cache.page_size, self.scale, window or 0, sinks)

    def seen(self, window=0, sinks=0):
        """[P, page_size]: the rows that anybody sees."""
        ps = self.cache.page_size
        seen = torch.zeros(self.cache.k.shape[0], ps, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            context = n - self.drafted[b]
            for t in range(self.drafted[b]):
                m = self.masks[b][t] & ((1 << self.drafted[b]) - 1)
                for j in range(n):
                    if drafted_reference.sees(j, context, m, window, sinks):
                        seen[self.table[b, j // ps], j % ps] = True
        return seen

    def given_back(self, window, sinks):
        """The table with the entries of pages that nobody sees out of range."""
        seen = self.seen(window, sinks).any(1)
        table = self.table.clone()
        for b, n in enumerate(self.lens):
            for i in range(-(-n // self.cache.page_size)):
                if not seen[table[b, i]]:
                    table[b, i] = BEHIND
        return table


CASES = [
    # lens, drafted, T, heads, group, page_size, d, query type, cache type, layout
    ([1], [1], 1, 1, 1, 16, 128, "bf16", "bf16", "phtd"),
    ([2, 17, 300], [2, 2, 2], 2, 2, 1, 16, 128, "bf16", "bf16", "pthd"),
    ([8, 129, 128, 500, 136], [8] * 5, 8, 2, 4, 16, 128, "bf16", "bf16", "phtd"),
    ([40, 0, 333, 5, 16], [13, 0, 16, 5, 16], 16, 1, 4, 64, 128, "bf16", "bf16", "kv"),
    ([64, 700, 257], [64] * 3, 64, 1, 4, 128, 128, "bf16", "bf16", "phtd"),
    ([300, 64], [64, 63], 64, 2, 2, 32, 64, "bf16", "bf16", "pthd"),
    ([500, 31], [31, 31], 31, 1, 8, 16, 128, "fp16", "fp16", "phtd"),
    ([200, 70], [5, 0], 5, 3, 5, 256, 64, "fp16", "fp16", "kv"),
    ([400, 8, 140], [8, 8, 8], 8, 2, 8, 16, 128, "bf16", "e4m3", "phtd"),
    ([400, 20, 140], [20, 7, 20], 20, 1, 3, 64, 64, "bf16", "e4m3", "pthd"),
    ([300, 64], [64, 64], 64, 1, 5, 32, 128, "bf16", "e4m3", "kv"),
    ([260, 20], [3, 3], 3, 2, 2, 16, 128, "fp16", "e4m3", "kv"),
    ([200, 90], [40, 40], 40, 1, 4, 128, 64, "fp16", "e4m3", "phtd"),
    ([200], [64], 64, 1, 16, 16, 64, "bf16", "bf16", "phtd"),
    ([30] * 40, [3] * 40, 3, 2, 3, 16, 64, "bf16", "bf16", "phtd"),
    ([0, 0], [0, 0], 4, 1, 2, 16, 128, "bf16", "bf16", "phtd"),
    ([1100, 1025], [9, 9], 9, 1, 1, 1024, 128, "bf16", "bf16", "phtd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_tree(cuda_device, case):
    s = Setup(*case, seed=len(case[0]) + case[2])
    check_tree(*s.run(), *s.want(), what=str(case))


@pytest.mark.parametrize("window,sinks", [(64, 0), (70, 3), (128, 128), (200, 140), (5000, 9)])
@pytest.mark.parametrize("case", [CASES[4], CASES[5], CASES[6], CASES[8], CASES[12], CASES[7]],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_tree_under_a_window(cuda_device, case, window, sinks):
    s = Setup(*case, seed=window + sinks)
    o, lse = s.run(s.given_back(window, sinks), window=window, sinks=sinks)
    check_tree(o, lse, *s.want(window, sinks), what=f"{case} {window} {sinks}")


@pytest.mark.parametrize("kind,q_type,T,group", [("bf16", "bf16", 5, 2), ("e4m3", "bf16", 7, 3),
                                                 ("fp16", "fp16", 40, 4), ("e4m3", "fp16", 60, 2)])
def test_short_windows_of_many_sequences(cuda_device, kind, q_type, T, group):
    """As many items as blocks, nearly: none is split, some are short."""
    rng = np.random.default_rng(T)
    lens = [int(n) for n in rng.integers(T, 1500, 70)]
    lens[:4] = [T, 1500, 0, T + 500]
    drafted = [min(n, T) for n in lens]
    drafted[5], drafted[6] = 0, 1
    s = Setup(lens, drafted, T, 2, group, 64, 64, q_type, kind, seed=T)
    window, sinks = 500, 6
    o, lse = s.run(window=window, sinks=sinks)
    for b in [0, 1, 2, 3, 5, 6, *range(7, 70, 8)]:
        context = lens[b] - drafted[b]
        assert (o[b, drafted[b]:] == 0).all() and (lse[b, drafted[b]:] == -math.inf).all()
        for t in range(0, drafted[b], 3):
            at = torch.tensor([j for j in range(lens[b]) if drafted_reference.sees(
                j, context, s.masks[b][t] & (1 << drafted[b]) - 1, window, sinks)])
            ids = s.table[b, at // 64].long()
            for h in range(2):
                k, v = (x[ids, h, at % 64] for x in (s.cache.k_values, s.cache.v_values))
                r = slice(h * group, (h + 1) * group)
                want = drafted_reference.ref.attend(s.q[b, t, r].double(), k, v, s.scale)
                check_tree(o[b, t, r], lse[b, t, r], *want, what=f"{b} {t} {h}")


@pytest.mark.parametrize("kind,q_type,T,group", [("bf16", "bf16", 5, 2), ("e4m3", "bf16", 7, 3),
                                                 ("fp16", "fp16", 40, 4), ("e4m3", "fp16", 60, 2)])
def test_longer_windows(cuda_device, kind, q_type, T, group):
    """Windows of several tiles of a few sequences: items are split, at any tile."""
    lens = [1500, 5000, T + 1290, T, 2600]
    drafted = [T, T - 1, T, T, T]
    s = Setup(lens, drafted, T, 2, group, 16, 64, q_type, kind, seed=T)
    for window, sinks in ((1200, 130), (1003, 0), (2500, 300)):
        o, lse = s.run(window=window, sinks=sinks)
        for b, n in enumerate(lens):
            context = n - drafted[b]
            for t in range(0, drafted[b], 2):
                at = torch.tensor([j for j in range(n) if drafted_reference.sees(
                    j, context, s.masks[b][t] & (1 << drafted[b]) - 1, window, sinks)])
                ids = s.table[b, at // 16].long()
                for h in range(2):
                    k, v = (x[ids, h, at % 16] for x in (s.cache.k_values, s.cache.v_values))
                    r = slice(h * group, (h + 1) * group)
                    want = drafted_reference.ref.attend(s.q[b, t, r].double(), k, v, s.scale)
                    check_tree(o[b, t, r], lse[b, t, r], *want, what=f"{window} {b} {t} {h}")


def test_masks_that_are_no_trees(cuda_device):
    """Rows that see nothing, only others, everything; bits from draft_lens on."""
    full = (1 << 64) - 1
    masks = [[0, 1 << 5, full, 0b1010101, 1, 1 << 63 | 1], [full] * 6, [0] * 6, [1 << 2] * 6]
    for lens in ([6, 6, 6, 6], [200, 100, 60, 6]):
        s = Setup(lens, [6, 4, 6, 2], 6, 2, 2, 16, 128, "bf16", "bf16", seed=1, masks=masks)
        o, lse = s.run()
        check_tree(o, lse, *s.want())
        assert (o[1, 4:] == 0).all() and (lse[1, 4:] == -math.inf).all()
    s = Setup([6, 6, 6, 6], [6, 4, 6, 2], 6, 2, 2, 16, 128, "bf16", "bf16", seed=1, masks=masks)
    o, lse = s.run()
    assert (o[2] == 0).all() and (lse[2] == -math.inf).all()  # no context, empty masks
    assert (o[3, 2:] == 0).all() and (lse[3, 2:] == -math.inf).all()  # (its context: 4 positions)
    check_tree(o, lse, *s.want())
    o, lse = s.run(window=6, sinks=1)
    check_tree(o, lse, *s.want(6, 1))


def test_one_tree_for_all_and_strides(cuda_device):
    s = Setup([100, 300], [7, 7], 7, 2, 2, 16, 128, "bf16", "bf16", seed=2)
    s.masks = [s.masks[0]] * 2
    want = s.run()
    q, k, v, table, lens, tree = s.args()
    got = fat.attn_tree_paged(q, k, v, table, lens, tree[0])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # heads outside the tokens, and rows of a wider table and mask
    turned = q.transpose(1, 2).contiguous().transpose(1, 2)
    big = torch.full((4, table.shape[1] + 3), BEHIND, dtype=torch.int32, device="cuda")
    big[::2, :table.shape[1]] = table
    masks = torch.full((2, 9), -1, dtype=torch.int64, device="cuda")
    masks[:, :7] = tree
    out = (torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"),
           torch.full(q.shape[:3], 7.0, device="cuda"))
    work = torch.empty(fat.attn_tree_workspace_bytes(2, 7, 4, 2, 128), dtype=torch.uint8,
                       device="cuda").fill_(255)
    got = fat.attn_tree_paged(turned, k, v, big[::2, :table.shape[1]], lens, masks[:, :7],
                              out=out, workspace=work)
    assert got[0] is out[0] and got[1] is out[1]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK


@pytest.mark.parametrize("kind,T,group", [("bf16", 9, 2), ("fp16", 9, 2), ("e4m3", 9, 2),
                                          ("bf16", 50, 4), ("e4m3", 50, 4), ("fp16", 50, 4)])
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
def test_what_nobody_sees_has_no_part(cuda_device, kind, T, group, fill):
    """Non-finite rows behind the sequences, in the gap of a window and in free pages."""
    s = Setup([300, 150, T + 1, T], [T, T - 3, 0, T], T, 2, group, 16, 128,
              "fp16" if kind == "fp16" else "bf16", kind, seed=3)
    want = s.run(window=70, sinks=5), s.run()
    for seen, window in ((s.seen(70, 5), dict(window=70, sinks=5)), (s.seen(), {})):
        hidden = ~seen[:, None, :, None].cuda().expand(s.cache.k.shape)
        for t in (s.cache.k, s.cache.v):
            keep = t.clone()
            if kind == "e4m3":
                t.view(torch.uint8)[hidden] = 0x7F
            else:
                t[hidden] = fill
            got = s.run(**window)
            assert all(torch.equal(a, b) for a, b in zip(got, want[0 if window else 1]))
            t.view(torch.uint8).copy_(keep.view(torch.uint8))


@pytest.mark.parametrize("kind,q_type", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"),
                                         ("e4m3", "fp16")])
@pytest.mark.parametrize("T,group", [(6, 2), (60, 4)])
def test_what_some_rows_do_not_see_has_no_part_in_them(cuda_device, kind, q_type, T, group):
    """A non-finite drafted token, or context position at a window's border, reaches the rows that
    see it and no other."""
    window, sinks = 64, 2
    lens = [T + 200, T + 65, 64 + T // 2]
    drafted = [T, T, T // 2]
    for fill in ((math.nan,) if kind == "e4m3" else (math.nan, math.inf, -math.inf)):
        s = Setup(lens, drafted, T, 1, group, 16, 128, q_type, kind, seed=4)
        ps = 16
        for b, n in enumerate(lens):
            context = n - drafted[b]
            # a drafted token, the border of the window, one position further in it
            for j in (context + 2, context - window + 2, context - window + 3):
                if j < 0:
                    continue
                page, at = int(s.table[b, j // ps]), j % ps
                if kind == "e4m3":
                    s.cache.scales[1][page, 0, at] = 255
                    s.cache.v_values[page, 0, at] = math.nan
                else:
                    s.cache.v[page, 0, at, 5 + j % 3] = fill
                    s.cache.v_values[page, 0, at, 5 + j % 3] = fill
        for w in (dict(window=window, sinks=sinks), {}):
            o, lse = s.run(**w)
            want = s.want(**w)
            magnitude = torch.where(torch.isfinite(want[2]), want[2], torch.zeros_like(want[2]))
            check_tree(o, lse, want[0], want[1], magnitude, what=f"{fill} {w}")
            assert torch.isfinite(want[0]).any() and not torch.isfinite(want[0]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
def test_keys_that_are_not_finite(cuda_device, kind):
    """A NaN key gives NaN to the rows that see it, and nothing to the others."""
    s = Setup([150, 80], [6, 6], 6, 1, 2, 16, 64, "fp16" if kind == "fp16" else "bf16", kind,
              seed=5)
    for b in range(2):
        j = s.lens[b] - 6 + 2
        page, at = int(s.table[b, j // 16]), j % 16
        if kind == "e4m3":
            s.cache.scales[0][page, 0, at] = 255
        else:
            s.cache.k[page, 0, at, 3] = math.nan
        s.cache.k_values[page, 0, at] = math.nan
    o, lse = s.run()
    want = s.want()
    check_tree(o, lse, want[0], want[1], torch.nan_to_num(want[2]))
    assert torch.isnan(want[0]).any() and torch.isfinite(want[0]).any()


def test_scores_far_apart(cuda_device):
    """Scores that rise by hundreds along the sequence, and fall: the running maximum moves at every
    tile.  (Times 40, so their error and the LSE's grow as much.)"""
    for kind, q_type in (("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")):
        for rising in (True, False):
            s = Setup([900, 600], [4, 4], 4, 1, 2, 64, 128, q_type, kind, seed=6)
            q = torch.randn(128, generator=torch.Generator().manual_seed(1))
            s.q[:] = (q / q.norm() * 11).to(s.q.dtype)
            for b, n in enumerate(s.lens):
                for j in range(n):
                    step = (j if rising else n - j) // 8 / 10.0
                    page, at = int(s.table[b, j // 64]), j % 64
                    row = (q / q.norm() * step * 5).to(s.cache.values[0].dtype)
                    if kind == "e4m3":
                        values, e = drafted_reference.ref.quantise_row(row.float().double().numpy())
                        s.cache.k_values[page, 0, at] = torch.tensor(values)
                        s.cache.scales[0][page, 0, at] = e
                        code = (torch.tensor(values) * 2.0 ** (127 - e)).float()
                        s.cache.k[page, 0, at] = code.to(torch.float8_e4m3fn).cuda()
                    else:
                        s.cache.k[page, 0, at] = row.to(TYPES[kind]).cuda()
                        s.cache.k_values[page, 0, at] = row.to(TYPES[kind]).double()
            check_tree(*s.run(), *s.want(), what=f"{kind} {rising}", grow=40)


@pytest.mark.parametrize("kind,q_type", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
def test_rows_of_unlike_magnitude(cuda_device, kind, q_type):
    """Values whose rows are up to 2^12 apart: what a small row adds is not lost beside what the
    sum of magnitudes allows."""
    s = Setup([500, 333], [7, 7], 7, 1, 3, 16, 64, q_type, kind, seed=7, spread=6)
    if kind != "e4m3":
        s.cache.k.copy_(s.cache.k.sign())  # (scores as assumed)
        s.cache.k_values.copy_(s.cache.k_values.sign())
    else:
        s.cache.scales[0].fill_(118)
        s.cache.k_values.copy_(s.cache.k.cpu().double() * 2.0 ** -9)
    check_tree(*s.run(), *s.want())


def test_one_sequence_across_all_blocks(cuda_device):
    """Long enough that every thread block gets part of it, and ragged ones."""
    for lens, T, group, kind in (([60000], 8, 4, "bf16"), ([20000, 9, 30000, 0, 700], 9, 2, "e4m3"),
                                 ([40000, 64], 64, 4, "bf16"), ([30000], 64, 3, "fp16")):
        drafted = [min(n, T) for n in lens]
        s = Setup(lens, drafted, T, 1, group, 64, 64, "fp16" if kind == "fp16" else "bf16", kind,
                  seed=8)
        o, lse = s.run()
        for b, n in enumerate(lens):  # (all rows of a sequence at once)
            if not n:
                assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
                continue
            ids = s.table[b, :-(-n // 64)].long()
            k, v = (x[ids, 0].reshape(-1, 64)[:n] for x in (s.cache.k_values, s.cache.v_values))
            for t in range(drafted[b]):
                at = torch.tensor([drafted_reference.sees(j, n - drafted[b], s.masks[b][t], 0, 0)
                                   for j in range(n - drafted[b], n)])
                at = torch.cat([torch.ones(n - drafted[b], dtype=torch.bool), at])
                want = drafted_reference.ref.attend(s.q[b, t].double(), k[at], v[at], s.scale)
                check_tree(o[b, t], lse[b, t], *want, what=f"{lens} {b} {t}")


def test_two_calls_give_the_same_bits(cuda_device):
    s = Setup([3000, 700, 64, 5000], [16] * 4, 16, 2, 4, 64, 128, "bf16", "bf16", seed=9)
    want = s.run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(s.run(), want))


def test_graphs_with_one_workspace(cuda_device):
    """Two captured calls, of unlike shapes, share a workspace; replays use the lengths, pages and
    trees of then."""
    a = Setup([2000, 300], [16, 16], 16, 2, 4, 64, 128, "bf16", "bf16", seed=10)
    b = Setup([900, 40, 1], [3, 3, 1], 3, 1, 2, 16, 64, "bf16", "e4m3", seed=11)
    work = torch.empty(max(fat.attn_tree_workspace_bytes(2, 16, 8, 2, 128),
                           fat.attn_tree_workspace_bytes(3, 3, 2, 1, 64)), dtype=torch.uint8,
                       device="cuda")
    calls, graphs, outs = [], [], []
    for s in (a, b):
        args, kw = s.args(), s.more(workspace=work)
        calls.append((args, kw))
        fat.attn_tree_paged(*args, **kw)
    torch.cuda.synchronize()
    for args, kw in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fat.attn_tree_paged(*args, **kw))
        graphs.append(graph)
    for turn in range(2):
        for s, (args, kw), graph, out in zip((a, b), calls, graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            check_tree(*out, *s.want())
        a.lens = [1500, 290]
        calls[0][0][4].copy_(torch.tensor(a.lens, dtype=torch.int32))
        a.masks = random_trees(2, 16, 77)
        calls[0][0][5].copy_(as_tensor(a.masks))
    assert fat.check_device_error() == fat.FAT_OK


def test_side_stream_and_its_memory(cuda_device):
    s = Setup([2000, 300], [16, 16], 16, 2, 4, 64, 128, "bf16", "bf16", seed=12)
    want = s.run()
    side = torch.cuda.Stream()
    args = s.args()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = fat.attn_tree_paged(*args, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_bad_indexes_are_reported(cuda_device):
    s = Setup([300, 200], [5, 5], 5, 2, 2, 16, 64, "bf16", "bf16", seed=13)
    good = s.run()
    for at, value in ((18, BEHIND), (18, -1), (0, 10 ** 6)):
        bad = s.table.clone()
        bad[0, at] = value
        o, _ = fat.attn_tree_paged(*s.args(bad))
        assert fat.check_device_error() == fat.FAT_ERR_INDEX
        assert torch.equal(o[1], good[0][1])
    for lens, drafted in (([-1, 200], None), ([10 ** 6, 200], None), ([4, 200], None),
                          ([300, 200], [6, 5]), ([300, 200], [-1, 5]), ([3, 200], [4, 5])):
        kw = {}
        if drafted:
            kw["draft_lens"] = torch.tensor(drafted, dtype=torch.int32).cuda()
        q, k, v, table, _, tree = s.args()
        o, _ = fat.attn_tree_paged(q, k, v, table, torch.tensor(lens, dtype=torch.int32).cuda(),
                                   tree, **kw)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX
        assert torch.equal(o[1], good[0][1])
    assert fat.check_device_error() == fat.FAT_OK


def test_refusals(cuda_device):
    s = Setup([300, 200], [5, 5], 5, 2, 2, 16, 64, "bf16", "bf16", seed=14)
    q, k, v, table, lens, tree = s.args()
    good = dict(q=q, k_cache=k, v_cache=v, page_table=table, seq_lens=lens, tree=tree)
    fat.attn_tree_paged(**good)
    for bad in (dict(q=q[:, 0]), dict(q=q.half()), dict(q=q[:1]), dict(q=q[:, :, :3]),
                dict(q=q[..., :32]), dict(q=q[:, :0], tree=tree[:, :0]),
                dict(q=q.repeat(1, 13, 1, 1), tree=tree.repeat(1, 13)),
                dict(tree=tree.int()), dict(tree=tree[:, :4]), dict(tree=tree[:1]),
                dict(tree=tree.T), dict(tree=None), dict(tree=tree.cpu()),
                dict(draft_lens=lens.long()), dict(draft_lens=lens[:1]),
                dict(draft_lens=torch.stack([lens, lens], 1)[:, 0]), dict(window=4),
                dict(window=2 ** 31), dict(window=0), dict(window=9, sinks=-1), dict(sinks=1),
                dict(out=(q, lens)), dict(workspace=lens), dict(seq_lens=lens[:1]),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            fat.attn_tree_paged(**{**good, **bad})
    with pytest.raises(ValueError, match="gradient"):
        fat.attn_tree_paged(**{**good, "q": q.clone().requires_grad_()})
    with pytest.raises(fat.FatError, match="INVALID_ARG"):
        fat.attn_tree_paged(**good, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros((2, 5, 4, 72), dtype=torch.bfloat16, device="cuda")[..., 4:68]
    with pytest.raises(fat.FatError, match="ALIGNMENT"):
        fat.attn_tree_paged(**{**good, "q": odd})
