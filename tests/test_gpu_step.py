"""Keeping accepted drafted tokens, and whole steps: prompts and drafted tokens are stored, judged
by tree attention, the accepted ones kept, and single tokens follow."""
import numpy as np
import pytest
import torch

import drafted_reference
import tensorized_online_softmax_gb300 as fat
from drafted_helpers import angle_table, as_tensor, check_tree, random_trees
from paged_helpers import BEHIND, TYPES, Cache, check_attention, make_table, pages_for

pytestmark = pytest.mark.gpu

CASES = [
    # context lengths, drafted, paths, heads, page_size, d, cache type, layout
    ([0, 30, 100], 8, [[0, 2, 7], [], [1]], 2, 16, 128, "bf16", "phtd"),
    ([5, 31], 20, [[0, 1, 2, 5, 6, 9, 10, 11, 13, 17, 19], list(range(20))], 3, 16, 64, "e4m3",
     "phtd"),
    ([63, 15, 40], 64, [[63], list(range(0, 64, 2)), list(range(64))], 1, 64, 128, "e4m3", "kv"),
    ([500], 40, [list(range(3, 40, 3))], 5, 32, 64, "fp16", "pthd"),
    # long paths, every row onto the one before it
    ([70, 3, 9], 400, [list(range(1, 300)), list(range(0, 400, 2)), list(range(399))], 2, 16, 128,
     "bf16", "phtd"),
    ([70, 16], 700, [list(range(1, 650)), list(range(30, 700))], 1, 16, 64, "e4m3", "pthd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-" + "-".join(map(str, c[3:])))
def test_keep(cuda_device, case):
    context, T, paths, heads, page_size, d, kind, layout = case
    lens = [n + T for n in context]
    cache = Cache(pages_for(lens, page_size), heads, page_size, d, kind, layout, seed=T)
    table = make_table(lens, page_size, cache.k.shape[0], seed=T)
    counts = [len(p) for p in paths]
    width = max(counts) + 2
    path = torch.full((len(context), width + 3), -5, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    want = [drafted_reference.keep(x.clone(), table, context, paths, counts, page_size)
            for x in cache.held()]
    fat.kv_cache_keep(cache.k, cache.v, table.cuda(),
                      torch.tensor(context, dtype=torch.int32).cuda(), path.cuda()[:, :width],
                      torch.tensor(counts, dtype=torch.int32).cuda(), **cache.scale_args)
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
    assert all(torch.equal(x, y) for x, y in zip(cache.held(), want))


def test_keep_reports_bad_entries(cuda_device):
    lens = [40, 40]
    cache = Cache(pages_for(lens, 16), 2, 16, 64, "e4m3", seed=1)
    table = make_table(lens, 16, cache.k.shape[0], width=3)
    table[0, 2] = table[1, 2] = BEHIND
    good = dict(context=[20, 20], path=[[1, 3], [0, 2]], counts=[2, 2])
    for bad in (dict(context=[-1, 20]), dict(context=[49, 20]), dict(context=[2 ** 31 - 1, 20]),
                dict(path=[[-3, -2], [0, 2]]), dict(path=[[1, 12], [0, 2]]),
                dict(path=[[1, 28], [0, 2]]), dict(path=[[1, 2 ** 31 - 1], [0, 2]]),
                dict(counts=[3, 2]), dict(counts=[-1, 2])):
        a = {**good, **bad}
        want = cache.held()
        if "counts" not in bad and "context" not in bad and a["path"][0][0] == 1:
            drafted_reference.keep(want[0], table, [20], [[1]], [1], 16)
            drafted_reference.keep(want[1], table, [20], [[1]], [1], 16)
        for x in want:
            drafted_reference.keep(x, table[1:], [20], [[0, 2]], [2], 16)
        fat.kv_cache_keep(cache.k, cache.v, table.cuda(),
                          *(torch.tensor(a[n], dtype=torch.int32).cuda()
                            for n in ("context", "path", "counts")), **cache.scale_args)
        assert fat.check_device_error() == fat.FAT_ERR_INDEX, bad
        assert all(torch.equal(x, y) for x, y in zip(cache.held(), want)), bad
    assert fat.check_device_error() == fat.FAT_OK


def test_keep_refusals(cuda_device):
    cache = Cache(5, 2, 16, 64, "bf16", seed=1)
    n = torch.tensor([3, 4], dtype=torch.int32).cuda()
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda()
    path = torch.tensor([[0, 1], [0, 2]], dtype=torch.int32).cuda()
    good = dict(k_cache=cache.k, v_cache=cache.v, page_table=table, context_lens=n, path=path,
                counts=n - 2)
    before = cache.held()
    fat.kv_cache_keep(**{**good, "path": path[:, :0]})
    assert all(torch.equal(x, y) for x, y in zip(cache.held(), before))
    for bad in (dict(path=path.long()), dict(path=path[:1]), dict(path=path[0]),
                dict(path=torch.stack([path, path], 2)[..., 0]), dict(counts=n[:1]),
                dict(counts=n.long()), dict(counts=torch.stack([n, n], 1)[:, 0]),
                dict(context_lens=n[:1]), dict(page_table=table.long()),
                dict(k_cache=cache.k[:1].expand(4, 2, 16, 64),
                     v_cache=cache.v[:1].expand(4, 2, 16, 64))):
        with pytest.raises(ValueError):
            fat.kv_cache_keep(**{**good, **bad})
    with pytest.raises(ValueError, match="gradient"):
        fat.kv_cache_keep(**{**good, "k_cache": cache.k.clone().requires_grad_()})


@pytest.mark.parametrize("kind,q_type,window", [("bf16", "bf16", None), ("e4m3", "bf16", 40),
                                                ("fp16", "fp16", 32)])
def test_steps(cuda_device, kind, q_type, window):
    """Prompt, two steps of drafted tokens, two single tokens: against the definitions over a list
    of rotated keys and values."""
    B, H, G, d, ps, T, sinks = 3, 2, 3, 64, 16, 6, 3 if window else 0
    g = torch.Generator().manual_seed(5)
    lens = [50, 7, 33]
    room = [n + 40 for n in lens]
    cache = Cache(pages_for(room, ps), H, ps, d, kind, seed=2)
    table = make_table(room, ps, cache.k.shape[0], seed=2)
    angles = angle_table(200, d)
    history = [[] for _ in range(B)]  # of each sequence the (k, v) that its positions hold, fp64
    dev = {"table": table.cuda(), "angles": angles.cuda()}

    def rows(n, heads):
        return torch.randn((n, heads, d), generator=g).to(TYPES[q_type])

    def stored(x):
        x = x.double()
        if kind == "e4m3":
            return drafted_reference.ref.quantise_rows(x)
        return x.float().to(TYPES[kind]).double()

    def append(new, depth):
        """new tokens of each sequence; their positions are the sequences' lengths + depth."""
        where = [(b, len(history[b]) + i) for b in range(B) for i in range(new[b])]
        at = [len(history[b]) + depth[b][i] for b in range(B) for i in range(new[b])]
        q, k, v = rows(len(where), H * G), rows(len(where), H), rows(len(where), H)
        slots = torch.tensor([int(table[b, j // ps]) * ps + j % ps for b, j in where])
        got = fat.kv_cache_append(q.cuda(), k.cuda(), v.cuda(), cache.k, cache.v, slots.cuda(),
                                  torch.tensor(at).cuda(), dev["angles"], **cache.scale_args)
        turned = drafted_reference.rotate(k.double(), angles.double(), [at], (d // 2,), False)
        for (b, _), kk, vv in zip(where, stored(turned), stored(v)):
            history[b].append((kk, vv))
        return got

    def values():
        """The caches that the history says, [P, H, page_size, d]."""
        k, v = torch.zeros((2,) + tuple(cache.k.shape), dtype=torch.float64)
        for b in range(B):
            for j, (kk, vv) in enumerate(history[b]):
                k[int(table[b, j // ps]), :, j % ps] = kk
                v[int(table[b, j // ps]), :, j % ps] = vv
        return k, v

    scale = float(np.float32(d ** -0.5))
    append(lens, [list(range(n)) for n in lens])
    for step in range(2):
        context = [len(h) for h in history]
        masks = random_trees(B, T, step)
        depth = [[bin(m).count("1") - 1 for m in line] for line in masks]
        q = append([T] * B, depth).view(B, T, H * G, d)
        n = torch.tensor([len(h) for h in history], dtype=torch.int32).cuda()
        o, lse = fat.attn_tree_paged(q, cache.k, cache.v, dev["table"], n, as_tensor(masks).cuda(),
                                     window=window, sinks=sinks, **cache.scale_args)
        k, v = values()
        want = drafted_reference.tree(q.cpu().double(), k, v, table, n.tolist(), [T] * B, masks,
                                      ps, scale, window or 0, sinks)
        # (keys rotated by the kernel are within a rounding of the history's: an e4m3 step of some
        # key moves a score by less than 2^-4 of |q||k| / sqrt(d): compared with what is held)
        held = cache.held()
        close = 2.0 ** -3 if kind == "e4m3" else 2.0 ** -7
        for b in range(B):
            for j in range(len(history[b])):
                a = held[0][int(table[b, j // ps]), :, j % ps]
                assert ((a - history[b][j][0]).abs() <=
                        close * a.abs() + 2.0 ** -8 * a.abs().amax()).all()
        want = drafted_reference.tree(q.cpu().double(), *held, table, n.tolist(), [T] * B, masks,
                                      ps, scale, window or 0, sinks)
        check_tree(o, lse, *want, what=f"step {step}")
        # a path from the root: a token, its parent, ... as rising indexes
        last = [T - 1, 0, T - 2]
        paths = [[t for t in range(T) if masks[b][last[b]] >> t & 1] for b in range(B)]
        path = torch.zeros((B, T), dtype=torch.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
        fat.kv_cache_keep(cache.k, cache.v, dev["table"],
                          torch.tensor(context, dtype=torch.int32).cuda(), path.cuda(),
                          counts.cuda(), **cache.scale_args)
        for b, p in enumerate(paths):
            history[b] = history[b][:context[b]] + [history[b][context[b] + t] for t in p]
    for step in range(2):
        q = append([1] * B, [[0]] * B)
        n = torch.tensor([len(h) for h in history], dtype=torch.int32).cuda()
        args = q, cache.k, cache.v, dev["table"], n
        o, lse = (fat.attn_decode_window(*args, window, sinks, **cache.scale_args) if window else
                  fat.attn_decode_paged(*args, **cache.scale_args))
        want = drafted_reference.window(q.cpu().double(), *cache.held(), table, n.tolist(), ps,
                                        scale, window or 10 ** 6, sinks)
        check_attention(o, lse, *want, what=f"token {step}", kind=kind)
        k, v = values()
        for b in range(B):  # the cache holds the history, accepted rows where they belong
            for j in range(len(history[b])):
                at = int(table[b, j // ps]), slice(None), j % ps
                assert torch.equal(cache.held()[1][at], v[at])
    torch.cuda.synchronize()
    assert fat.check_device_error() == fat.FAT_OK
