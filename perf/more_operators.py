"""Cases that measure the operators of a speculative decoding step over the paged cache.

The cache: keys and values in pages, ``[pages, kv_heads, page_size, head_dim]``, as bf16, fp16, or
e4m3 codes with one power-of-two scale per row (a uint8 exponent byte e, the row's value being
code * 2^(e - 127)).  ``page_table[b, i]`` is the page of positions [i * page_size,
(i + 1) * page_size) of sequence b, whose length is ``seq_lens[b]``.  Kinds of case:

``append``  the newest tokens' queries and keys are rotated by their positions (a table of cosines
            and sines; one position axis, or time, height and width), keys and values are stored in
            the cache; an e4m3 cache is read back as [B, H, N, d], the others come back as they are
``tree``    drafted tokens, the last positions of every sequence, attend to its context and to
            those drafted tokens that a mask of bits allows (their ancestors in a tree)
``window``  one new query token per sequence attends to the last positions of its sequence and to a
            few first ones
``keep``    drafted tokens are appended, then the rows of the accepted path are moved to the
            positions right behind the context

Where ``own`` is false the operators run in their plain form (elementary torch operations in 32
bits), where it is true as calls of the framework.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- the cases
def _case(name, kind, batch, kv_heads, group, head_dim, page_size, len_min, len_max, q_type,
          cache_type, tokens=1, window=0, sinks=0, ragged=False, rotated=0, axes=1,
          interleaved=False):
    c = dict(kind=kind, batch=batch, kv_heads=kv_heads, group=group, head_dim=head_dim,
             page_size=page_size, len_min=len_min, len_max=len_max, q_type=q_type,
             cache_type=cache_type, tokens=tokens, window=window, sinks=sinks, ragged=ragged,
             rotated=rotated, axes=axes, interleaved=interleaved)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decoding step of young sequences: one token each, all latency
        _case("append_step", "append", 16, 8, 4, 128, 16, 1, 64, "bf16", "e4m3", rotated=128),
        # prompts with images: positions of three axes, every token new
        _case("append_prompts", "append", 6, 8, 4, 128, 64, 1000, 8192, "bf16", "bf16", 8192,
              rotated=128, axes=3),
        # one short chat with a few drafted tokens: the smallest call
        _case("tree_one_short", "tree", 1, 8, 4, 128, 16, 208, 208, "bf16", "bf16", 8),
        # an ordinary batch: 16 drafted tokens, 64 query rows to a cached head
        _case("tree_batch16", "tree", 16, 8, 4, 128, 64, 1000, 8192, "bf16", "bf16", 16),
        # the widest trees: 256 query rows to a cached head
        _case("tree_wide", "tree", 8, 8, 4, 128, 128, 4096, 16384, "bf16", "bf16", 64),
        # a large batch over a quantised cache
        _case("tree_e4m3_batch32", "tree", 32, 8, 8, 128, 64, 4096, 16384, "bf16", "e4m3", 8),
        # head dim 64, one query head per cached head, a padded batch, a window with sinks
        _case("tree_fp16_d64_odd", "tree", 13, 20, 1, 64, 32, 5, 4097, "fp16", "fp16", 5,
              window=1024, sinks=4, ragged=True),
        # one short chat under a window: latency
        _case("window_one_short", "window", 1, 8, 4, 128, 16, 700, 700, "bf16", "bf16",
              window=512, sinks=4),
        # long contexts, of which each token sees 4096 positions and four sinks
        _case("window_batch32", "window", 32, 8, 4, 128, 64, 8192, 32768, "bf16", "bf16",
              window=4096, sinks=4),
        # short windows over very long sequences in a quantised cache, small pages, odd sizes
        _case("window_e4m3_page16", "window", 48, 8, 8, 128, 16, 50000, 131072, "bf16", "e4m3",
              window=1000, sinks=65),
        # a step's drafted tokens are stored, the accepted path is kept
        _case("keep_step", "keep", 4, 8, 4, 128, 16, 20, 100, "bf16", "e4m3", 8, rotated=128),
        # the same for a large batch of the widest trees
        _case("keep_batch64", "keep", 64, 8, 4, 128, 64, 100, 2048, "bf16", "bf16", 64,
              rotated=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "tree", "tree", "window", "keep"])
    d = rng.choice([64, 128])
    kv_heads = _log_int(rng, 1, 24)
    group = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    page_size = rng.choice([16, 32, 64, 128, 256])
    batch = _log_int(rng, 1, 64)
    q_type = rng.choice(["bf16", "bf16", "fp16"])
    cache_type = rng.choice([q_type, "e4m3"])
    heads = batch * kv_heads * d
    tokens, window, sinks, ragged, rotated, axes, inter = 1, 0, 0, False, 0, 1, False
    if kind in ("append", "keep"):
        most = (1 << 24) if kind == "append" else (1 << 23)
        len_max = _log_int(rng, 17, max(64, min(8192 if kind == "append" else 1024,
                                                most // (heads * (group + 1)))))
        tokens = rng.choice([1, _log_int(rng, 1, len_max), len_max]) if kind == "append" \
            else _log_int(rng, 1, min(64, len_max))
        rotated = rng.choice([d, d, d // 2, 32])
        axes = rng.choice([1, 1, 3])
        inter = rng.choice([False, False, True])
    elif kind == "tree":
        tokens = _log_int(rng, 1, 64)
        most = min((1 << 28) // heads, (1 << 27) // (batch * kv_heads * group * tokens))
        len_max = _log_int(rng, max(17, tokens), max(128, min(32768, most)))
        ragged = rng.choice([False, True])
        if rng.random() < 0.4:
            window, sinks = tokens + _log_int(rng, 1, 2048), rng.choice([0, 1, 4, 70])
    else:
        window, sinks = _log_int(rng, 1, 4096), rng.choice([0, 1, 4, 16, 130])
        while heads * (window + sinks) > 1 << 27:
            window = window // 2 + 1
        len_max = _log_int(rng, 17, 131072)
    len_min = rng.choice([0, 1, len_max // 3, len_max // 2, len_max])
    if kind in ("tree", "keep"):
        len_min = max(len_min, 0 if ragged else tokens)
    return _case(None, kind, batch, kv_heads, group, d, page_size, len_min, len_max, q_type,
                 cache_type, tokens, window, sinks, ragged, rotated, axes, inter)


def _lens(c):
    """The sequences' lengths and how many of their positions are new: fixed by the case."""
    rng = random.Random("%d %d %d" % (c["batch"], c["len_min"], c["len_max"]))
    lens = [c["len_max"]] + [rng.randint(c["len_min"], c["len_max"])
                             for _ in range(c["batch"] - 1)]
    new = [min(n, c["tokens"]) for n in lens]
    if c["ragged"]:
        new = [new[0]] + [rng.randint(0, n) for n in new[1:]]
    return lens, new


def _accepted(c):
    """How many drafted tokens of each sequence are accepted in a ``keep`` case."""
    rng = random.Random("%d %d" % (c["batch"], c["tokens"]))
    return [rng.randint(1, min(c["tokens"], 12)) for _ in range(c["batch"])]


def _seen(c):
    """For each sequence the ranges of positions that any of its rows sees."""
    lens, new = _lens(c)
    ranges = []
    for n, t in zip(lens, new):
        if not c["window"]:
            ranges.append([(0, n)])
        else:
            lo = max(0, (n - t if c["kind"] == "tree" else n - 1) + 1 - c["window"])
            s = min(c["sinks"], n)
            ranges.append([(0, n)] if s >= lo else [(0, s), (lo, n)])
    return ranges


def work(case):
    c = case
    lens, new = _lens(c)
    ps, d, H, G, B = (c[x] for x in ("page_size", "head_dim", "kv_heads", "group", "batch"))
    q8 = c["cache_type"] == "e4m3"
    row = d * (1 if q8 else 2) + (1 if q8 else 0)  # one cached row, K or V
    if c["kind"] in ("append", "keep"):
        n = sum(new)
        heads = n * (2 * H * G * d * 2 + 2 * H * d * 2 + 2 * H * row)
        total = heads + n * (8 + 8 * c["axes"]) + 4 * c["rotated"] * min(n, max(lens))
        if c["kind"] == "keep":
            total += sum(_accepted(c)) * (4 * H * row + 4) + 8 * B
        if q8:  # read back
            total += 2 * sum(lens) * H * row + 2 * B * H * max(lens) * d * 2
        return {"bytes": total, "flops": 3 * n * H * (G + 1) * c["rotated"]}
    seen = [sum(b - a for a, b in r) for r in _seen(c)]
    pages = sum(sum(-(-b // ps) - a // ps for a, b in r if b > a) for r in _seen(c))
    rows = B * H * G * (c["tokens"] if c["kind"] == "tree" else 1)
    per = new if c["kind"] == "tree" else [1] * B
    return {"bytes": 2 * sum(seen) * H * row + rows * (4 * d + 4) + 4 * (pages + B)
            + (8 * B * c["tokens"] if c["kind"] == "tree" else 0),
            "flops": 4 * H * G * d * sum(s * t for s, t in zip(seen, per))}


# ------------------------------------------------------------- e4m3 rows
def _power(e):
    """2^(e - 127) as fp32 for exponent bytes e (1..254); NaN for 255."""
    p = (e.to(torch.int32) << 23).view(torch.float32)
    return torch.where(e == 255, torch.full_like(p, float("nan")), p)


def _quantise(x):
    """fp32 rows -> (e4m3 codes, exponent bytes): the least power of two that brings the row's
    largest magnitude to at most 448; a row of zeros has scale 1, one with inf or NaN byte 255."""
    top = x.abs().amax(-1)
    bits = top.view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    e = torch.where(top == 0, torch.full_like(e, 127), e.clamp(min=1))
    good = torch.isfinite(x).all(-1)
    e = torch.where(good, e, torch.full_like(e, 255))
    inverse = ((254 - e.clamp(max=253)) << 23).view(torch.float32)
    scaled = torch.where(good[..., None], x * inverse[..., None],
                         torch.full_like(x, float("nan")))
    return scaled.to(torch.float8_e4m3fn), e.to(torch.uint8)


def _rows_of(cache, scale, page, at):
    """fp32 values of single rows: page and at of any shape -> [*shape, H, d]."""
    if scale is None:
        return cache[page, :, at].float()
    codes = cache.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn)
    return codes.float() * _power(scale[page, :, at])[..., None]


def _sequences(cache, scale, table, n):
    """The first n positions of every sequence in fp32: [B, H, n, d]."""
    ps, H, d = cache.shape[2], cache.shape[1], cache.shape[3]
    ids = table[:, :-(-n // ps)].long()
    if scale is None:
        x = cache[ids].float()
    else:
        codes = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn)
        x = codes.float() * _power(scale[ids])[..., None]
    return x.permute(0, 2, 1, 3, 4).reshape(table.shape[0], H, -1, d)[:, :, :n]


# --------------------------------------------------------------- the inputs
def _sections(c):
    """How many of the rotated pairs belong to each position axis."""
    pairs = c["rotated"] // 2
    if c["axes"] == 1:
        return (pairs,)
    part = 3 * pairs // 8
    return (pairs - 2 * part, part, part)


def prepare(case, seed):
    c = dict(case)
    lens, new = _lens(c)
    ps, d, H, G, B = (c[x] for x in ("page_size", "head_dim", "kv_heads", "group", "batch"))
    q8 = c["cache_type"] == "e4m3"
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    pick = random.Random(int(seed))
    typ, ctyp = TYPES[c["q_type"]], TYPES[c["cache_type"]]
    # pages are held for what can still be seen; the others have been given back
    held = [sorted({i for a, b in r for i in range(a // ps, -(-b // ps))}) for r in _seen(c)]
    counts = [-(-n // ps) for n in lens]
    used, width = sum(len(x) for x in held), max(1, max(counts))
    pool = used + used // 10 + 1
    # pages in the order in which an allocator hands them out after some churn
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    # entries behind a sequence's pages, and of pages given back, hold pages of somebody else
    table = torch.randint(0, pool, (B, width), generator=g, device=dev, dtype=torch.int32)
    where = torch.tensor([b * width + i for b, x in enumerate(held) for i in x],
                         dtype=torch.int64, device=dev)
    table.view(-1)[where] = order[:used]
    # keys have channels of unlike size, as projections with a learned bias and scale give
    channel = torch.exp(0.5 * torch.randn((H, 1, d), generator=g, device=dev))
    st = {"case": c, "lens": lens, "new": new, "table": table, "max_len": max(lens),
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    for name in ("k", "v"):
        cache = torch.empty((pool, H, ps, d), dtype=ctyp, device=dev)
        scale = torch.empty((pool, H, ps), dtype=torch.uint8, device=dev) if q8 else None
        step = max(1, (1 << 27) // (H * ps * d))
        for a in range(0, pool, step):  # in pieces: the fp32 values need four times the room
            n = min(step, pool - a)
            x = torch.randn((n, H, ps, d), generator=g, device=dev)
            x = x * channel if name == "k" else x
            if q8:
                codes, e = _quantise(x)
                cache.view(torch.uint8)[a:a + n] = codes.view(torch.uint8)
                scale[a:a + n] = e
            else:
                cache[a:a + n] = x.to(ctyp)
        st[name + "_cache"], st[name + "_scale"] = cache, scale
    if c["kind"] == "window":
        st["q"] = torch.randn((B, H * G, d), generator=g, device=dev).to(typ)
        return st
    T = c["tokens"]
    if c["kind"] == "tree":
        st["q"] = torch.randn((B, T, H * G, d), generator=g, device=dev).to(typ)
        # a drafted token's parent is an earlier one, or (-1) the context's last token
        st["parents"] = [[-1] + [pick.randint(max(-1, t - 6), t - 1) for t in range(1, T)]
                         for _ in range(B)]
        masks = []
        for line in st["parents"]:
            m = []
            for t, p in enumerate(line):
                m.append((m[p] if p >= 0 else 0) | 1 << t)
            masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        st["tree"] = torch.tensor(masks, dtype=torch.int64, device=dev)
        st["draft_lens"] = torch.tensor(new, dtype=torch.int32, device=dev) if c["ragged"] else None
        return st
    which = [(b, p) for b, n in enumerate(lens) for p in range(n - new[b], n)]
    w = torch.tensor(which, dtype=torch.int64, device=dev).reshape(-1, 2)
    st["slots"] = table[w[:, 0], w[:, 1] // ps].long() * ps + w[:, 1] % ps
    at = w[:, 1]
    st["positions"] = at if c["axes"] == 1 else torch.stack([at // 64, at % 64 // 8, at % 8])
    pairs = c["rotated"] // 2
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)
    angle = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * freq
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    for name, heads in (("q", H * G), ("k", H), ("v", H)):
        x = torch.randn((len(which), heads, d), generator=g, device=dev)
        st[name] = (x * channel[:, 0] if name == "k" else x).to(typ)
    if c["kind"] == "keep":
        st["accepted"] = [min(a, n) for a, n in zip(_accepted(c), new)]
        st["paths"] = [sorted(pick.sample(range(n), a)) for a, n in zip(st["accepted"], new)]
        M = max(st["accepted"])
        st["path"] = torch.tensor([x + [0] * (M - len(x)) for x in st["paths"]],
                                  dtype=torch.int32, device=dev)
        st["counts"] = torch.tensor(st["accepted"], dtype=torch.int32, device=dev)
        st["base"] = torch.tensor([n - t for n, t in zip(lens, new)], dtype=torch.int32,
                                  device=dev)
    return st


# ----------------------------------------------------------- the plain forms
def _rotate(st, x):
    """x [tokens, heads, d] in fp32, rotated by its tokens' positions."""
    c = st["case"]
    n = c["rotated"]
    rows = st["cos_sin"][st["positions"]]  # [(axes,) tokens, n]
    if c["axes"] == 1:
        cos, sin = rows[:, :n // 2], rows[:, n // 2:]
    else:
        parts = [x.split(_sections(c), -1) for x in (rows[..., :n // 2], rows[..., n // 2:])]
        cos, sin = (torch.cat([part[a][a] for a in range(c["axes"])], -1) for part in parts)
    cos, sin = cos[:, None], sin[:, None]
    if c["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., n:]], -1)


def _plain_append(st):
    ps = st["case"]["page_size"]
    page, at = st["slots"] // ps, st["slots"] % ps
    for name in ("k", "v"):
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        x = st[name].float()
        x = _rotate(st, x) if name == "k" else x
        if scale is None:
            cache[page, :, at] = x.to(cache.dtype)
        else:
            codes, e = _quantise(x)
            cache.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            scale[page, :, at] = e
    return _rotate(st, st["q"].float()).to(st["q"].dtype)


def _plain_read(st):
    """The caches themselves, or what a quantised one holds."""
    if st["k_scale"] is None:
        return st["k_cache"], st["v_cache"]
    out = []
    live = torch.arange(st["max_len"], device=st["table"].device) < st["seq_lens"][:, None]
    for name in ("k", "v"):
        x = _sequences(st[name + "_cache"], st[name + "_scale"], st["table"], st["max_len"])
        out.append(torch.where(live[:, None, :, None], x, 0.0).to(st[name].dtype))
    return tuple(out)


def _plain_keep(st):
    ps = st["case"]["page_size"]
    i = torch.arange(st["path"].shape[1], device=st["path"].device)
    base = st["base"].long()[:, None]
    to = base + i
    # (what is not accepted is copied onto itself)
    source = torch.where(i < st["counts"][:, None], base + st["path"].long(), to)
    to, source = to.clamp(max=st["max_len"] - 1), source.clamp(max=st["max_len"] - 1)
    table = st["table"].long()
    live = i < st["counts"][:, None]
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        x = st[name]
        if x is None:
            continue
        x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        rows = x[table.gather(1, source // ps), :, source % ps]
        # rows past the accepted ones go where the first one goes, with its value
        keep = live.reshape(live.shape + (1,) * (rows.dim() - 2))
        x[table.gather(1, torch.where(live, to, base) // ps), :,
          torch.where(live, to, base) % ps] = torch.where(keep, rows, rows[:, :1])


def _softmax(s, v):
    """Scores s (-inf where nothing is seen) against values v: (o, LSE); zeros for empty rows."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v)
    return torch.where(total == 0, torch.zeros_like(o), o / total), (m + torch.log(total))[..., 0]


def _plain_tree(st):
    c, n, T = st["case"], st["max_len"], st["case"]["tokens"]
    B, H, G, d = (c[x] for x in ("batch", "kv_heads", "group", "head_dim"))
    k = _sequences(st["k_cache"], st["k_scale"], st["table"], n)
    v = _sequences(st["v_cache"], st["v_scale"], st["table"], n)
    dev = k.device
    length = st["seq_lens"].long()[:, None, None]
    drafted = torch.full_like(length, T) if st["draft_lens"] is None \
        else st["draft_lens"].long()[:, None, None]
    context = length - drafted
    bits = st["tree"][:, :, None] >> torch.arange(T, device=dev) & 1  # [B, T, T]
    bits = bits * (torch.arange(T, device=dev) < drafted)
    at = torch.arange(n, device=dev)
    inside = (at >= context) & (at < length)  # [B, 1, n]
    mine = bits.gather(2, (at - context).clamp(0, T - 1).expand(B, T, n)) > 0
    before = (at < context).expand(B, T, n)
    if c["window"]:
        here = context + bits.sum(-1, keepdim=True) - 1  # the position of each drafted token
        before = before & ((at < c["sinks"]) | (at > here - c["window"]))
    live = (before | (inside & mine)) & (torch.arange(T, device=dev)[:, None] < drafted)
    q = st["q"].view(B, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d).float()
    s = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    s = s.view(B, H, T, G, n).masked_fill(~live[:, None, :, None], -math.inf)
    v = torch.where((at < length[:, 0])[:, None, :, None], v, 0.0)
    o, lse = _softmax(s.view(B, H, T * G, n), v)
    o = o.view(B, H, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, H * G, d)
    return o.to(st["q"].dtype), lse.view(B, H, T, G).transpose(1, 2).reshape(B, T, H * G)


def _plain_window(st):
    c = st["case"]
    B, H, G, d, ps = (c[x] for x in ("batch", "kv_heads", "group", "head_dim", "page_size"))
    dev = st["table"].device
    n = st["seq_lens"].long()[:, None]
    W = min(c["window"], st["max_len"])
    S = min(c["sinks"], st["max_len"])
    first = torch.arange(S, device=dev).expand(B, S)
    last = n - W + torch.arange(W, device=dev)
    at = torch.cat([first, last], 1)  # the positions seen, the sinks among the last ones once
    live = torch.cat([first < n, last >= S], 1)
    at = at.clamp(0, st["max_len"] - 1)
    page = st["table"].long().gather(1, at // ps)
    k, v = (_rows_of(st[x + "_cache"], st[x + "_scale"], page, at % ps).transpose(1, 2)
            for x in ("k", "v"))
    s = torch.matmul(st["q"].view(B, H, G, d).float(), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    s = torch.where(live[:, None, None], s, -math.inf)
    o, lse = _softmax(s, torch.where(live[:, None, :, None], v, 0.0))
    return o.to(st["q"].dtype).flatten(1, 2), lse.flatten(1)


# --------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    if own:
        import tensorized_online_softmax_gb300 as fat

        kw = {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
        if c["kind"] == "tree":
            more = {"window": c["window"], "sinks": c["sinks"]} if c["window"] else {}
            return fat.attn_tree_paged(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                       st["seq_lens"], st["tree"], draft_lens=st["draft_lens"],
                                       **more, **kw)
        if c["kind"] == "window":
            return fat.attn_decode_window(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                          st["seq_lens"], c["window"], c["sinks"], **kw)
        q = fat.kv_cache_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                st["slots"], st["positions"], st["cos_sin"],
                                sections=_sections(c) if c["axes"] > 1 else None,
                                interleaved=c["interleaved"], **kw)
        if c["kind"] == "keep":
            fat.kv_cache_keep(st["k_cache"], st["v_cache"], st["table"], st["base"], st["path"],
                              st["counts"], **kw)
        if st["k_scale"] is None:
            return q, st["k_cache"], st["v_cache"]
        return (q,) + tuple(fat.kv_cache_read(st["k_cache"], st["v_cache"], st["table"],
                                              st["seq_lens"], st["max_len"],
                                              dtype=st["k"].dtype, **kw))
    if c["kind"] == "tree":
        return _plain_tree(st)
    if c["kind"] == "window":
        return _plain_window(st)
    q = _plain_append(st)
    if c["kind"] == "keep":
        _plain_keep(st)
    return (q,) + tuple(_plain_read(st))


# ------------------------------------------------------- the definition, in 64 bits
def _row_values(x):
    """What rows x (fp64) hold after e4m3 storage with a power-of-two scale: the nearest
    multiple of each value's step, ties to the even multiple (no inf or NaN in the cases)."""
    top = x.abs().amax(-1, keepdim=True)
    tiny = torch.finfo(torch.float64).tiny
    s = torch.ceil(torch.log2(top.clamp(min=tiny) / 448)).clamp(min=-126)
    s = torch.where(top > 448 * torch.exp2(s), s + 1, s)
    s = torch.where(top <= 448 * torch.exp2(s - 1), s - 1, s).clamp(min=-126)
    s = torch.where(top == 0, torch.zeros_like(s), s)
    binade = torch.frexp(x.abs())[1].double() - 1
    step = torch.exp2(torch.maximum(binade - 3, s - 9))
    return torch.round(x / step) * step


def _wide(cache, scale, ids):
    x = cache.view(torch.uint8)[ids].view(cache.dtype).double() if scale is not None \
        else cache[ids].double()
    return x if scale is None else torch.ldexp(x, scale[ids].int().double()[..., None] - 127)


def _walk(st, name, b, at):
    """The positions `at` (a list) of sequence b in fp64: [H, len(at), d]."""
    ps = st["case"]["page_size"]
    at = torch.as_tensor(at, dtype=torch.int64, device=st["table"].device)
    pages, back = torch.unique(at // ps, return_inverse=True)
    x = _wide(st[name + "_cache"], st[name + "_scale"], st["table"][b, pages].long())
    return x.transpose(0, 1).flatten(1, 2)[:, back * ps + at % ps]


def _turned(st, x):
    """x [tokens, heads, d] in fp64 as complex numbers times the table's unit ones."""
    c = st["case"]
    n, pairs = c["rotated"], c["rotated"] // 2
    table = torch.complex(st["cos_sin"][:, :pairs].double(), st["cos_sin"][:, pairs:].double())
    axis = [a for a, count in enumerate(_sections(c)) for _ in range(count)]
    where = st["positions"].view(c["axes"], -1)
    turn = torch.stack([table[where[a], i] for i, a in enumerate(axis)], -1)[:, None]
    y = x.double().clone()
    lo = slice(0, n, 2) if c["interleaved"] else slice(0, pairs)
    hi = slice(1, n, 2) if c["interleaved"] else slice(pairs, n)
    z = torch.complex(y[..., lo], y[..., hi]) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_append(st):
    c, lens, new = st["case"], st["lens"], st["new"]
    ps, H, d, B = (c[x] for x in ("page_size", "kv_heads", "head_dim", "batch"))
    out = [_turned(st, st["q"])]
    first = [sum(new[:b]) for b in range(B)]
    for name in ("k", "v"):
        x = _turned(st, st["k"]) if name == "k" else st["v"].double()
        quantised = st[name + "_scale"] is not None
        x = _row_values(x) if quantised else x
        if quantised:
            full = torch.zeros((B, H, max(lens), d), dtype=torch.float64, device=x.device)
            for b, n in enumerate(lens):
                if n:
                    full[b, :, :n] = _walk(st, name, b, list(range(n)))
        else:
            full = st[name + "_cache"].double()
        for b, n in enumerate(lens):
            rows = x[first[b]:first[b] + new[b]].clone()
            if c["kind"] == "keep":
                rows[:st["accepted"][b]] = x[[first[b] + i for i in st["paths"][b]]]
            if quantised:
                full[b, :, n - new[b]:n] = rows.transpose(0, 1)
                continue
            at = torch.arange(n - new[b], n, device=x.device)
            full[st["table"][b, at // ps].long(), :, at % ps] = rows
        out.append(full)
    return tuple(out)


def _softmax_attention(q, k, v):
    """q [H, G, d], k, v [H, n, d], all fp64."""
    if k.shape[1] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=q.dtype,
                                               device=q.device)
    s = (q @ k.mT) / math.sqrt(q.shape[-1])
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)


def exact(case, seed):
    st = prepare(case, seed)
    c, lens, new = st["case"], st["lens"], st["new"]
    H, G, d, B, T = (c[x] for x in ("kv_heads", "group", "head_dim", "batch", "tokens"))
    if c["kind"] in ("append", "keep"):
        return _exact_append(st)
    dev = st["table"].device
    if c["kind"] == "window":
        q = st["q"].double().view(B, H, G, d)
        o, lse = torch.empty_like(q), torch.empty((B, H, G), dtype=q.dtype, device=dev)
        for b, n in enumerate(lens):
            seen = [j for a, e in _seen(c)[b] for j in range(a, e)]
            o[b], lse[b] = _softmax_attention(q[b], _walk(st, "k", b, seen),
                                              _walk(st, "v", b, seen))
        return o.flatten(1, 2), lse.flatten(1)
    q = st["q"].double().view(B, T, H, G, d)
    o = torch.zeros((B, T, H, G, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, T, H, G), -math.inf, dtype=torch.float64, device=dev)
    for b, (n, drafted) in enumerate(zip(lens, new)):
        context = n - drafted
        if not drafted:
            continue
        seen = [j for a, e in _seen(c)[b] for j in range(a, e)]
        k, v = _walk(st, "k", b, seen), _walk(st, "v", b, seen)
        place = torch.tensor(seen, device=dev)
        hidden = torch.empty((drafted, len(seen)), dtype=torch.bool)
        for t in range(drafted):
            line, p = [], t
            while p >= 0:
                line.append(p)
                p = st["parents"][b][p]
            here = context + len(line) - 1
            low = here - c["window"] + 1 if c["window"] else 0
            ok = (place < context) & ((place < c["sinks"]) | (place >= low))
            ok |= torch.isin(place, torch.tensor([context + p for p in line], device=dev))
            hidden[t] = ~ok.cpu()
        s = torch.einsum("thgd,hnd->htgn", q[b, :drafted], k) / math.sqrt(d)
        s = s.masked_fill(hidden.to(dev)[None, :, None], -math.inf)
        o[b, :drafted] = torch.einsum("htgn,hnd->thgd", torch.softmax(s, -1), v)
        lse[b, :drafted] = torch.logsumexp(s, -1).transpose(0, 1)
    return o.flatten(2, 3), lse.flatten(2, 3)
