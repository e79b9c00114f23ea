"""Cases that measure the serving operators over a paged key-value cache.

The cache: keys and values in pages, ``[pages, kv_heads, page_size, head_dim]``,
as bf16, fp16, or e4m3 codes with one power-of-two scale per row (a uint8
exponent byte e, the row's value being code * 2^(e - 127); 255 marks a row
that holds an inf or NaN and reads as NaN).  ``page_table[b, i]`` is the page
of positions [i * page_size, (i + 1) * page_size) of sequence b, whose length
is ``seq_lens[b]``.  Kinds of case:

``cache``   the newest tokens of every sequence are written to the cache (and
            quantised, e4m3), then the sequences are read back as [B, H, N, d]
``decode``  one new query token per sequence attends to its cached sequence
``score``   the bounds (elementwise minimum and maximum of the keys) of the
            blocks that the newest token touched are renewed, then every block
            of every sequence gets its score: an upper bound on q . k
``sparse``  one new query token per sequence attends to the blocks with the
            highest scores (one block is one page)

Where ``own`` is false the operators run in their plain form (elementary torch
operations in 32 bits), where it is true as calls of the framework.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- the cases
def _case(name, kind, batch, kv_heads, group, head_dim, page_size, len_min, len_max, q_type,
          cache_type, new_tokens=1, num_blocks=0):
    c = dict(kind=kind, batch=batch, kv_heads=kv_heads, group=group, head_dim=head_dim,
             page_size=page_size, len_min=len_min, len_max=len_max, q_type=q_type,
             cache_type=cache_type, new_tokens=new_tokens, num_blocks=num_blocks)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decoding step of a few young sequences stores its token: all latency
        _case("cache_e4m3_step", "cache", 4, 8, 1, 128, 16, 1, 64, "bf16", "e4m3", 1),
        # whole prompts go into a quantised cache and come back for the prompt's attention
        _case("cache_e4m3_prompts", "cache", 6, 8, 1, 128, 64, 1000, 8192, "bf16", "e4m3", 8192),
        # chunked prefill without quantisation: 1024 new tokens, the prefix read back with them
        _case("cache_fp16_chunk", "cache", 3, 12, 1, 64, 32, 5000, 20000, "fp16", "fp16", 1024),
        # one short chat: the smallest call
        _case("decode_one_short", "decode", 1, 8, 4, 128, 16, 200, 200, "bf16", "bf16"),
        # an ordinary batch of ragged sequences, grouped heads
        _case("decode_batch32", "decode", 32, 8, 4, 128, 64, 1000, 8192, "bf16", "bf16"),
        # one very long document: few rows, a long axis
        _case("decode_one_long", "decode", 1, 8, 4, 128, 128, 131072, 131072, "bf16", "bf16"),
        # a large batch over a quantised cache
        _case("decode_e4m3_batch64", "decode", 64, 8, 8, 128, 64, 4096, 16384, "bf16", "e4m3"),
        # one query head per cached head, head dim 64, odd counts, an empty slot in the batch
        _case("decode_fp16_d64_odd", "decode", 13, 20, 1, 64, 32, 0, 4097, "fp16", "fp16"),
        # block scores of a batch with long contexts, and of small pages over a quantised cache
        _case("score_batch16", "score", 16, 8, 4, 128, 64, 16384, 32768, "bf16", "bf16"),
        _case("score_e4m3_page16", "score", 16, 8, 8, 128, 16, 32768, 65536, "bf16", "e4m3"),
        # attention over the best 64 of up to 512 blocks
        _case("sparse_batch16", "sparse", 16, 8, 4, 128, 64, 16384, 32768, "bf16", "bf16",
              num_blocks=64),
        # two very long sequences, small pages, many blocks, a quantised cache
        _case("sparse_e4m3_page16", "sparse", 2, 4, 16, 128, 16, 100000, 131072, "bf16", "e4m3",
              num_blocks=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["cache", "decode", "decode", "score", "sparse"])
    d = rng.choice([64, 128])
    kv_heads = _log_int(rng, 1, 24)
    group = rng.choice([1, 1, 2, 3, 4, 5, 8, 16]) if kind != "cache" else 1
    page_size = rng.choice([16, 32, 64, 128, 256])
    batch = _log_int(rng, 1, 96)
    # elements of the cached keys: no drawn case is larger than the largest listed one
    most = {"cache": 1 << 25, "decode": 1 << 29, "score": 1 << 28, "sparse": 1 << 28}[kind]
    longest = max(64, min(131072, most // (batch * kv_heads * d)))
    len_max = _log_int(rng, 17, longest)
    len_min = rng.choice([0, 1, len_max // 3, len_max // 2, len_max])
    q_type = rng.choice(["bf16", "bf16", "fp16"])
    cache_type = rng.choice([q_type, "e4m3"])
    new_tokens = rng.choice([1, _log_int(rng, 1, len_max), len_max]) if kind == "cache" else 1
    num_blocks = _log_int(rng, 1, 600) if kind == "sparse" else 0
    return _case(None, kind, batch, kv_heads, group, d, page_size, len_min, len_max, q_type,
                 cache_type, new_tokens, num_blocks)


def _lens(c):
    """The sequences' lengths: fixed by the case, the first one the longest."""
    rng = random.Random("%d %d %d" % (c["batch"], c["len_min"], c["len_max"]))
    return [c["len_max"]] + [rng.randint(c["len_min"], c["len_max"])
                             for _ in range(c["batch"] - 1)]


def work(case):
    c = case
    lens, ps, d = _lens(c), c["page_size"], c["head_dim"]
    H, G, B = c["kv_heads"], c["group"], c["batch"]
    q8 = c["cache_type"] == "e4m3"
    row = d * (1 if q8 else 2) + (1 if q8 else 0)  # one cached row, K or V
    tokens, pages = sum(lens), sum(-(-n // ps) for n in lens)
    index = 4 * (pages + B)
    if c["kind"] == "cache":
        new = sum(min(n, c["new_tokens"]) for n in lens)
        out = 2 * B * H * max(lens) * d * 2
        return {"bytes": new * (8 + 2 * H * d * 2 + 2 * H * row) + 2 * tokens * H * row + out
                + index, "flops": 0}
    heads = 2 * B * H * G * (2 * d) + 4 * B * H * G  # q, o and the LSE
    if c["kind"] == "decode":
        return {"bytes": 2 * tokens * H * row + heads + index, "flops": 4 * tokens * H * G * d}
    if c["kind"] == "score":
        last = sum((n - 1) % ps + 1 for n in lens if n)
        return {"bytes": last * H * row + 2 * pages * H * d * 2 + pages * H * 4
                + B * H * G * d * 2 + index + sum(1 for n in lens if n) * H * 2 * d * 2,
                "flops": 4 * pages * H * G * d}
    chosen = sum(min(-(-n // ps), c["num_blocks"]) * ps - (-n % ps) for n in lens if n)
    return {"bytes": 2 * chosen * H * row + heads + 4 * pages * H + 4 * B * H * c["num_blocks"]
            + index, "flops": 4 * chosen * H * G * d}


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


def _pages_of(cache, scale, ids):
    """fp32 values of the pages `ids`: [*ids.shape, H, page_size, d]."""
    if scale is None:
        return cache[ids].float()
    codes = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    return codes.float() * _power(scale[ids])[..., None]


def _sequences(cache, scale, table, n):
    """The first n positions of every sequence in fp32: [B, H, n, d]."""
    ps, H, d = cache.shape[2], cache.shape[1], cache.shape[3]
    x = _pages_of(cache, scale, table[:, :-(-n // ps)].long())
    return x.permute(0, 2, 1, 3, 4).reshape(table.shape[0], H, -1, d)[:, :, :n]


# --------------------------------------------------------------- the inputs
def prepare(case, seed):
    c = dict(case)
    lens, ps, d = _lens(c), c["page_size"], c["head_dim"]
    H, G, B = c["kv_heads"], c["group"], c["batch"]
    q8 = c["cache_type"] == "e4m3"
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    typ, ctyp = TYPES[c["q_type"]], TYPES[c["cache_type"]]
    counts = [-(-n // ps) for n in lens]
    used, width = sum(counts), max(counts)
    pool = used + used // 10 + 1
    # pages in the order in which an allocator hands them out after some churn
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    # entries behind a sequence's pages hold pages of somebody else
    table = torch.randint(0, pool, (B, width), generator=g, device=dev, dtype=torch.int32)
    start = torch.tensor([sum(counts[:b]) for b in range(B)], device=dev)
    col = torch.arange(width, device=dev)
    inside = col[None, :] < torch.tensor(counts, device=dev)[:, None]
    table = torch.where(inside, order[(start[:, None] + col[None, :]).clamp(max=pool - 1)], table)
    # keys have channels of unlike size, as projections with a learned bias and scale give
    channel = torch.exp(0.5 * torch.randn((H, 1, d), generator=g, device=dev))

    def rows(n, scale_by):
        return torch.randn((n, H, ps, d), generator=g, device=dev) * scale_by

    st = {"case": c, "lens": lens, "table": table, "max_len": max(lens),
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    for name in ("k", "v") if c["kind"] != "score" else ("k",):
        cache = torch.empty((pool, H, ps, d), dtype=ctyp, device=dev)
        scale = torch.empty((pool, H, ps), dtype=torch.uint8, device=dev) if q8 else None
        step = max(1, (1 << 27) // (H * ps * d))
        for a in range(0, pool, step):  # in pieces: the fp32 values need four times the room
            n = min(step, pool - a)
            x = rows(n, channel if name == "k" else 1.0)
            if q8:
                codes, e = _quantise(x)
                cache.view(torch.uint8)[a:a + n] = codes.view(torch.uint8)
                scale[a:a + n] = e
            else:
                cache[a:a + n] = x.to(ctyp)
        st[name + "_cache"], st[name + "_scale"] = cache, scale
    if c["kind"] == "cache":
        which = [(b, p) for b, n in enumerate(lens) for p in range(max(0, n - c["new_tokens"]), n)]
        w = torch.tensor(which, dtype=torch.int64, device=dev).reshape(-1, 2)
        st["slots"] = table[w[:, 0], w[:, 1] // ps].long() * ps + w[:, 1] % ps
        for name in ("k", "v"):
            by = channel[:, 0] if name == "k" else 1.0
            st[name] = (torch.randn((len(which), H, d), generator=g, device=dev) * by).to(typ)
        return st
    st["q"] = torch.randn((B, H * G, d), generator=g, device=dev).to(typ)
    if c["kind"] == "score":
        bounds = torch.empty((pool, H, 2, d), dtype=typ, device=dev)
        step = max(1, (1 << 27) // (H * ps * d))
        for a in range(0, pool, step):
            ids = torch.arange(a, min(a + step, pool), device=dev)
            x = _pages_of(st["k_cache"], st["k_scale"], ids)
            bounds[ids] = torch.stack([x.amin(2), x.amax(2)], 2).to(typ)
        st["bounds"] = bounds
    if c["kind"] == "sparse":
        st["scores"] = torch.randn((B, H, width), generator=g, device=dev) * 4
    return st


# ----------------------------------------------------------- the plain forms
def _plain_cache(st):
    ps = st["case"]["page_size"]
    page, at = st["slots"] // ps, st["slots"] % ps
    out = []
    for name in ("k", "v"):
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        if scale is None:
            cache[page, :, at] = st[name]
        else:
            codes, e = _quantise(st[name].float())
            cache.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            scale[page, :, at] = e
        x = _sequences(cache, scale, st["table"], st["max_len"])
        live = torch.arange(st["max_len"], device=x.device) < st["seq_lens"][:, None]
        out.append(torch.where(live[:, None, :, None], x, 0.0).to(st[name].dtype))
    return tuple(out)


def _attend(q, k, v, live):
    """q [B, H, G, d] against k, v [B, H, n, d] where `live` [B, H or 1, n]; (o, LSE)."""
    s = torch.matmul(q.float(), k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    s = torch.where(live[:, :, None, :], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(live[..., None], v, 0.0))
    o = torch.where(total == 0, torch.zeros_like(o), o / total)  # no key at all: zeros
    return o.to(q.dtype).flatten(1, 2), (m + torch.log(total)).flatten(1)


def _plain_decode(st):
    c, n = st["case"], st["max_len"]
    k = _sequences(st["k_cache"], st["k_scale"], st["table"], n)
    v = _sequences(st["v_cache"], st["v_scale"], st["table"], n)
    live = torch.arange(n, device=k.device) < st["seq_lens"][:, None]
    q = st["q"].view(c["batch"], c["kv_heads"], c["group"], c["head_dim"])
    return _attend(q, k, v, live[:, None, :])


def _plain_score(st):
    c, bounds, table, n = st["case"], st["bounds"], st["table"], st["seq_lens"].long()
    ps, H, G, d = c["page_size"], c["kv_heads"], c["group"], c["head_dim"]
    last = (n - 1).clamp(min=0)
    page = table.long().gather(1, (last // ps)[:, None])[:, 0]
    x = _pages_of(st["k_cache"], st["k_scale"], page)  # [B, H, ps, d]
    live = (torch.arange(ps, device=x.device) <= (last % ps)[:, None])[:, None, :, None]
    low = torch.where(live, x, math.inf).amin(2)
    high = torch.where(live, x, -math.inf).amax(2)
    fresh = torch.stack([low, high], 2).to(bounds.dtype)
    bounds[page] = torch.where((n > 0)[:, None, None, None], fresh, bounds[page])
    lo_hi = bounds[table.long()].float()  # [B, width, H, 2, d]
    q = st["q"].view(-1, H, G, d).float()
    s = torch.einsum("bhgd,bwhd->bhgw", q.clamp(min=0), lo_hi[..., 1, :])
    s = s + torch.einsum("bhgd,bwhd->bhgw", q.clamp(max=0), lo_hi[..., 0, :])
    s = s.amax(2)
    blocks = (n + ps - 1) // ps
    inside = torch.arange(table.shape[1], device=s.device) < blocks[:, None]
    return bounds, torch.where(inside[:, None, :], s, -math.inf)


def _plain_sparse(st):
    c, scores, table = st["case"], st["scores"], st["table"]
    ps, H, G, d = c["page_size"], c["kv_heads"], c["group"], c["head_dim"]
    B, width, take = c["batch"], table.shape[1], min(c["num_blocks"], table.shape[1])
    n = st["seq_lens"].long()
    count = ((n + ps - 1) // ps)[:, None, None]
    at = torch.arange(width, device=scores.device)
    # highest score first, the lower index first among equals; the newest block before all
    # others and nothing past the end
    order = torch.sort(scores, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    rank = torch.where(at == count - 1, -1, torch.where(at < count, rank, width))
    order = torch.sort(rank, dim=-1, stable=True).indices[..., :take]
    order = torch.where(rank.gather(-1, order) < width, order, width)
    chosen = torch.sort(order, dim=-1).values  # ascending; `width` where there is none
    some = chosen < width
    blocks = torch.full((B, H, c["num_blocks"]), -1, dtype=torch.int32, device=scores.device)
    blocks[..., :take] = torch.where(some, chosen, -1)
    pages = table.long()[torch.arange(B, device=at.device)[:, None, None],
                         chosen.clamp(max=width - 1)]
    head = torch.arange(H, device=at.device)[None, :, None]

    def rows(cache, scale):
        if scale is None:
            x = cache[pages, head].float()
        else:
            codes = cache.view(torch.uint8)[pages, head].view(torch.float8_e4m3fn)
            x = codes.float() * _power(scale[pages, head])[..., None]
        return x.reshape(B, H, take * ps, d)

    place = chosen[..., None] * ps + torch.arange(ps, device=at.device)
    live = (some[..., None] & (place < n[:, None, None, None])).reshape(B, H, take * ps)
    o, lse = _attend(st["q"].view(B, H, G, d), rows(st["k_cache"], st["k_scale"]),
                     rows(st["v_cache"], st["v_scale"]), live)
    return o, lse, blocks


# --------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    if own:
        import tensorized_online_softmax_gb300 as fat

        kw = {"k_scale": st["k_scale"]}
        if c["kind"] == "score":
            bounds = fat.kv_block_bounds(st["k_cache"], st["table"], st["seq_lens"],
                                         st["bounds"], 1, **kw)
            return bounds, fat.kv_block_scores(st["q"], bounds, st["table"], st["seq_lens"],
                                               c["page_size"])
        kw["v_scale"] = st["v_scale"]
        if c["kind"] == "cache":
            fat.kv_cache_write(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], **kw)
            return fat.kv_cache_read(st["k_cache"], st["v_cache"], st["table"], st["seq_lens"],
                                     st["max_len"], dtype=st["k"].dtype, **kw)
        if c["kind"] == "decode":
            return fat.attn_decode_paged(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                         st["seq_lens"], **kw)
        return fat.attn_decode_sparse(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                      st["seq_lens"], st["scores"], c["num_blocks"], **kw)
    return {"cache": _plain_cache, "decode": _plain_decode, "score": _plain_score,
            "sparse": _plain_sparse}[c["kind"]](st)


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


def _walk(st, name, b, n):
    """Positions 0..n-1 of sequence b in fp64: [H, n, d]."""
    ps = st["case"]["page_size"]
    x = _wide(st[name + "_cache"], st[name + "_scale"], st["table"][b, :-(-n // ps)].long())
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _softmax_attention(q, k, v):
    """One sequence: q [H, G, d], k, v [H, n, d], all fp64."""
    if k.shape[1] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=q.dtype,
                                               device=q.device)
    s = (q @ k.mT) / math.sqrt(q.shape[-1])
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)


def exact(case, seed):
    st = prepare(case, seed)
    c, lens = st["case"], st["lens"]
    ps, H, G, d, B = (c[x] for x in ("page_size", "kv_heads", "group", "head_dim", "batch"))
    dev = st["table"].device
    if c["kind"] == "cache":
        out = []
        for name in ("k", "v"):
            x = st[name].double()
            x = _row_values(x) if st[name + "_scale"] is not None else x
            full = torch.zeros((B, H, max(lens), d), dtype=torch.float64, device=dev)
            row = 0
            for b, n in enumerate(lens):
                new = min(n, c["new_tokens"])
                if n:
                    full[b, :, :n] = _walk(st, name, b, n)
                    full[b, :, n - new:n] = x[row:row + new].transpose(0, 1)
                row += new
            out.append(full)
        return tuple(out)
    q = st["q"].double().view(B, H, G, d)
    if c["kind"] == "score":
        bounds = st["bounds"].double()
        scores = torch.full((B, H, st["table"].shape[1]), -math.inf, dtype=torch.float64,
                            device=dev)
        for b, n in enumerate(lens):
            if n:
                rows = _wide(st["k_cache"], st["k_scale"],
                             st["table"][b, (n - 1) // ps].long())[:, :(n - 1) % ps + 1]
                bounds[st["table"][b, (n - 1) // ps].long()] = torch.stack(
                    [rows.min(1).values, rows.max(1).values], 1)
        for b, n in enumerate(lens):
            blocks = -(-n // ps)
            for a in range(0, blocks, 512):
                w = bounds[st["table"][b, a:min(a + 512, blocks)].long()]  # [w, H, 2, d]
                w = w.permute(1, 2, 0, 3)[:, :, None]  # [H, 2, 1, w, d]
                qq = q[b][:, :, None, :]
                best = torch.where(qq >= 0, qq * w[:, 1], qq * w[:, 0]).sum(-1)
                scores[b, :, a:min(a + 512, blocks)] = best.max(1).values
        return bounds, scores
    o = torch.empty((B, H, G, d), dtype=torch.float64, device=dev)
    lse = torch.empty((B, H, G), dtype=torch.float64, device=dev)
    for b, n in enumerate(lens):
        if c["kind"] == "decode":
            o[b], lse[b] = _softmax_attention(q[b], _walk(st, "k", b, n), _walk(st, "v", b, n))
            continue
        if n == 0:
            o[b], lse[b] = 0, -math.inf
            continue
        k, v, blocks = _walk(st, "k", b, n), _walk(st, "v", b, n), -(-n // ps)
        table = st["scores"][b].tolist()
        for h in range(H):
            best = sorted(range(blocks - 1), key=lambda j: (-table[h][j], j))
            best = sorted(best[:c["num_blocks"] - 1] + [blocks - 1])
            keep = torch.cat([torch.arange(j * ps, min(n, (j + 1) * ps)) for j in best]).to(dev)
            o[b, h:h + 1], lse[b, h:h + 1] = _softmax_attention(
                q[b, h:h + 1], k[h:h + 1, keep], v[h:h + 1, keep])
    o, lse = o.flatten(1, 2), lse.flatten(1)
    return (o, lse) if c["kind"] == "decode" else (o, lse, None)
