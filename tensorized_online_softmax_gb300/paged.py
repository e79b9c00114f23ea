"""Serving over a paged key-value cache: the binding of the ``fat_kv_*`` and
``fat_attn_decode_*`` entry points of ``include/fat_attn.h``.

The cache is two tensors ``k_cache, v_cache`` of shape ``[num_pages, heads,
page_size, d]`` (any order of the first three dimensions in memory: pass a
transposed view), bf16, fp16 or ``torch.float8_e4m3fn``; an e4m3 cache has one
scale byte per row beside it, ``k_scale, v_scale``: contiguous uint8
``[num_pages, heads, page_size]``, the row's values being
``code * 2**(byte - 127)`` and 255 marking a row with an inf or NaN.
``page_table`` (int32 ``[B, width]``) gives the page of positions
``[i * page_size, (i + 1) * page_size)`` of each sequence, ``seq_lens`` (int32
``[B]``) the sequences' lengths.  Both live on the device, so a page or length
out of range cannot be refused here: the kernels skip it, and
:func:`check_device_error` then returns ``FAT_ERR_INDEX``.

Every call is asynchronous on ``stream`` (default: torch's current stream of
the tensors' device), and allocates its outputs and workspace unless they are
given, from that stream's memory: they need no wait for the current stream.
(Inputs, and outputs that are given, are the caller's to order.)  A given workspace must not be shared by calls that overlap.  Calls can
be captured in a graph (after a first call of their kind, which loads the
kernels); replays use the lengths, pages and slots that the tensors hold then.
Nothing here is differentiable: a tensor that requires a gradient is refused
unless gradients are off (``torch.no_grad()``, ``torch.inference_mode()``).
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import DTYPES, FatError, _empty, _given, load_library

_P, _I, _L, _F, _Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float,
                      ctypes.c_size_t)


# The structs go to the library as packed bytes (half the time of a ctypes struct); the classes
# mirror them for whoever calls the C entry points directly.
class FatKvCache(ctypes.Structure):
    """Mirror of ``fat_kv_cache`` in include/fat_attn.h (same field order)."""
    _fields_ = [
        ("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P),
        ("num_pages", _L), ("heads", _I), ("page_size", _I), ("d", _I), ("dtype", _I),
        ("k_page_stride", _L), ("k_head_stride", _L), ("k_token_stride", _L),
        ("v_page_stride", _L), ("v_head_stride", _L), ("v_token_stride", _L),
    ]


class FatPageTable(ctypes.Structure):
    """Mirror of ``fat_page_table`` in include/fat_attn.h (same field order)."""
    _fields_ = [("pages", _P), ("stride", _L), ("width", _I), ("batch", _I), ("seq_lens", _P)]


_pack_cache = struct.Struct("@PPPPqiiiiqqqqqq").pack
_pack_table = struct.Struct("@PqiiP").pack


def declare(lib) -> None:
    """Argument and result types of the entry points used here."""
    cache = table = _P
    query = [_P, _I, _L, _L, _I]
    for name, args, result in (
            ("fat_kv_write", [cache, _P, _P, _I, _L, _L, _L, _L, _P, _I, _P], _I),
            ("fat_kv_read", [cache, table, _P, _P, _I, _I, _P], _I),
            ("fat_attn_decode_paged", [cache, table, *query, _F, _P, _P, _P, _Z, _P], _I),
            ("fat_attn_decode_workspace_bytes", [_I, _I, _I, _I], _Z),
            ("fat_kv_block_bounds", [cache, table, _I, _P, _I, _P], _I),
            ("fat_kv_block_scores", [*query, _P, _L, _I, _I, _I, table, _P, _P], _I),
            ("fat_attn_decode_sparse",
             [cache, table, *query, _P, _I, _I, _I, _F, _P, _P, _P, _P, _Z, _P], _I),
            ("fat_attn_decode_sparse_workspace_bytes", [_I, _I, _I, _I, _I], _Z)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, result


_WIDE = {torch.bfloat16: DTYPES["bf16"], torch.float16: DTYPES["fp16"]}
_CACHE = {**_WIDE, torch.float8_e4m3fn: DTYPES["e4m3"]}
_E4M3 = DTYPES["e4m3"]
_MOST = 1 << 30  # of counts that the C interface takes (and ctypes would cut to 32 bits)
_DIRECT = 512  # FAT_DECODE_DIRECT: positions of a table that need no workspace

# The checks below run for every call of a serving loop, where a few microseconds count: each
# function first asks everything at once, and only finds out what is wrong if something is.


def _wrong(name, t, dtypes, dim, device=None):
    """Raises if a tensor is not what `dtypes`, `dim` and `device` say."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, not {t.dim()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _tensor(name, t, dtypes, dim, device=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == dim
            and (device is None or t.device == device)):
        _wrong(name, t, dtypes, dim, device)
    return t


def _gradient():
    """Some argument requires a gradient, which would be lost without a word."""
    if torch.is_grad_enabled():
        raise ValueError("no gradient flows through the paged operators: call them under "
                         "torch.no_grad(), or detach what requires one")


def _rows(name, t, pages, heads, writable):
    """Strides between pages, heads and tokens; those of a dimension of one entry do not matter (a
    page has 16 rows at least)."""
    a, b, c, row = t.stride()
    if row != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if pages == 1:
        a = 0
    if heads == 1:
        b = 0
    if writable and ((a == 0 and pages > 1) or (b == 0 and heads > 1) or c == 0):
        raise ValueError(f"{name} is a broadcast view: its rows share memory")
    return a, b, c


def _scale(name, t, shape, device):
    if t is None:
        raise ValueError(f"an e4m3 cache needs {name}")
    _tensor(name, t, (torch.uint8,), 3, device)
    if t.shape != shape[:3] or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [num_pages, heads, page_size]")
    return t.data_ptr()


def _cache(k, v, k_scale, v_scale, writable=False):
    """The checked cache, v None where only the keys are read: the packed struct, the device, the
    fat_dtype, and (pages, heads, page_size, d)."""
    if not (isinstance(k, torch.Tensor) and k.is_cuda and k.dim() == 4 and k.dtype in _CACHE):
        _wrong("k_cache", k, _CACHE, 4)
    device, dtype, shape = k.device, k.dtype, k.shape
    kind = _CACHE[dtype]
    pages, heads, page_size, d = shape
    k_rows = _rows("k_cache", k, pages, heads, writable)
    if v is None:
        at, v_rows = 0, (0, 0, 0)
    else:
        if not (isinstance(v, torch.Tensor) and v.device == device and v.dtype is dtype
                and v.shape == shape):
            _wrong("v_cache", v, (dtype,), 4, device)
            raise ValueError("k_cache and v_cache must have the same shape")
        at, v_rows = v.data_ptr(), _rows("v_cache", v, pages, heads, writable)
    if k.requires_grad or (at and v.requires_grad):
        _gradient()
    ks = vs = 0
    if kind == _E4M3:
        ks = _scale("k_scale", k_scale, shape, device)
        vs = _scale("v_scale", v_scale, shape, device) if v is not None else 0
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales go with an e4m3 cache only")
    return _pack_cache(k.data_ptr(), at, ks, vs, pages, heads, page_size, d, kind, *k_rows,
                       *v_rows), device, kind, shape


def _table(page_table, seq_lens, device):
    """The checked table as a packed struct, the batch and the entries of a sequence."""
    if not (isinstance(page_table, torch.Tensor) and isinstance(seq_lens, torch.Tensor)
            and page_table.device == seq_lens.device == device
            and page_table.dtype is seq_lens.dtype is torch.int32
            and page_table.dim() == 2 and seq_lens.dim() == 1):
        _wrong("page_table", page_table, (torch.int32,), 2, device)
        _wrong("seq_lens", seq_lens, (torch.int32,), 1, device)
    batch, width = page_table.shape
    stride, step = page_table.stride()
    if seq_lens.shape[0] != batch or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be contiguous [B], page_table [B, width]")
    if step != 1 and width > 1:
        raise ValueError("the rows of page_table must be contiguous")
    return _pack_table(page_table.data_ptr(), stride if batch > 1 else width, width, batch,
                       seq_lens.data_ptr()), batch, width


def _query(q, batch, heads, d, device):
    """q [B, Hq, d] -> its pointer, type, strides and head count as C arguments."""
    if not (isinstance(q, torch.Tensor) and q.device == device and q.dim() == 3
            and q.dtype in _WIDE):
        _wrong("q", q, _WIDE, 3, device)
    b, h, c = q.shape
    if q.requires_grad:
        _gradient()
    if b != batch or c != d or h < 1 or h % heads:
        raise ValueError(f"q must be [{batch}, a multiple of {heads}, {d}], "
                         f"not {list(q.shape)}")
    per_batch, per_head, step = q.stride()
    if step != 1:
        raise ValueError("the rows of q must be contiguous")
    return (q.data_ptr(), _WIDE[q.dtype], per_batch if b > 1 else 0, per_head if h > 1 else 0, h)


def _tokens(name, t, shape, dtypes, device):
    """k or v [T, heads, d] -> its strides between tokens and heads."""
    _tensor(name, t, dtypes, 3, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    a, b, row = t.stride()
    if row != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return a if shape[0] > 1 else 0, b if shape[1] > 1 else 0


def _output(name, t, shape, dtype, device):
    _tensor(name, t, (dtype,), len(shape), device)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {list(shape)}")
    if t.requires_grad:
        _gradient()
    return t


def _handle(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None \
        else stream.cuda_stream


def _call(name, device, *args):
    """The library's function on the tensors' device."""
    fn = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status:
        raise FatError(status, name)


def kv_cache_write(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None,
                   stream=None) -> None:
    """Store new tokens in a paged cache, quantising them if it is e4m3.

    ``k, v``: [T, heads, d], bf16 or fp16 (the cache's own type unless it is
    e4m3); strided views are fine if every row starts on 16 bytes.  ``slots``:
    int64 [T], ``page * page_size + place`` of each token; a negative slot
    skips the token.  The slots of one call must differ.  An e4m3 row gets the
    least power of two as its scale that brings its largest magnitude to at
    most 448.
    """
    cache, device, kind, (_, heads, _, d) = _cache(k_cache, v_cache, k_scale, v_scale, True)
    _tensor("slots", slots, (torch.int64,), 1, device)
    shape = (slots.shape[0], heads, d)
    k_strides = _tokens("k", k, shape, _WIDE, device)
    v_strides = _tokens("v", v, shape, (k.dtype,), device)
    if kind != _E4M3 and k.dtype != k_cache.dtype:
        raise ValueError(f"a {k_cache.dtype} cache takes {k_cache.dtype} tokens, not {k.dtype}")
    if k.requires_grad or v.requires_grad:
        _gradient()
    if not shape[0]:
        return
    if shape[0] > 0x7fffffff:
        raise ValueError("more than 2^31 - 1 tokens in one call")
    if not slots.is_contiguous():
        raise ValueError("slots must be contiguous")
    _call("fat_kv_write", device, cache, k.data_ptr(), v.data_ptr(), _WIDE[k.dtype], *k_strides,
          *v_strides, slots.data_ptr(), shape[0], _handle(_given(stream, device), device))


def kv_cache_read(k_cache, v_cache, page_table, seq_lens, max_len: int, *, dtype=None,
                  k_scale=None, v_scale=None, out=None, stream=None):
    """Read cached sequences back: ``(k, v)``, contiguous [B, heads, max_len, d].

    ``dtype``: bf16 or fp16; the cache's own type (the default) unless it is
    e4m3 (default bf16).  Rows from a sequence's length on are zeros.
    """
    cache, device, kind, (_, heads, _, d) = _cache(k_cache, v_cache, k_scale, v_scale)
    table, batch, _ = _table(page_table, seq_lens, device)
    if dtype is None:
        dtype = torch.bfloat16 if kind == _E4M3 else k_cache.dtype
    if dtype not in _WIDE or (kind != _E4M3 and dtype != k_cache.dtype):
        raise ValueError(f"a {k_cache.dtype} cache is not read as {dtype}")
    shape = (batch, heads, int(max_len), d)
    if not 1 <= shape[2] <= _MOST:
        raise ValueError("max_len must be 1 to 2^30")
    stream = _given(stream, device)
    if out is None:
        k, v = (_empty(shape, dtype, device, stream) for _ in range(2))
    else:
        k, v = (_output(n, x, shape, dtype, device) for n, x in zip(("k", "v"), out))
    _call("fat_kv_read", device, cache, table, k.data_ptr(), v.data_ptr(), _WIDE[dtype], shape[2],
          _handle(stream, device))
    return k, v


def _decode_arguments(q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, out, stream):
    cache, device, kind, shape = _cache(k_cache, v_cache, k_scale, v_scale)
    table, batch, width = _table(page_table, seq_lens, device)
    query = _query(q, batch, shape[1], shape[3], device)
    if kind != _E4M3 and q.dtype != k_cache.dtype:
        raise ValueError(f"a {k_cache.dtype} cache takes {k_cache.dtype} queries, not {q.dtype}")
    stream = _given(stream, device)
    if out is None and stream is None:  # (the quickest way to the same)
        o = torch.empty_like(q) if q.is_contiguous() else q.new_empty(q.shape)
        lse = q.new_empty((batch, query[4]), dtype=torch.float32)
    elif out is None:
        o = _empty(q.shape, q.dtype, device, stream)
        lse = _empty((batch, query[4]), torch.float32, device, stream)
    else:
        o = _output("o", out[0], q.shape, q.dtype, device)
        lse = _output("lse", out[1], (batch, query[4]), torch.float32, device)
    return (cache, table, *query), device, shape, batch, width, o, lse, stream


@functools.lru_cache(maxsize=256)
def attn_decode_workspace_bytes(batch: int, q_heads: int, kv_heads: int, d: int,
                                num_blocks: int | None = None) -> int:
    """Workspace size of :func:`attn_decode_paged`, or with ``num_blocks`` of
    :func:`attn_decode_sparse` (0 for invalid arguments)."""
    lib = load_library()
    if num_blocks is None:
        return lib.fat_attn_decode_workspace_bytes(batch, q_heads, kv_heads, d)
    return lib.fat_attn_decode_sparse_workspace_bytes(batch, q_heads, kv_heads, d, num_blocks)


def _workspace(workspace, sizes, device, stream):
    """The workspace's address and size; allocated if not given."""
    if workspace is None:
        nbytes = attn_decode_workspace_bytes(*sizes)
        return _empty((nbytes,), torch.uint8, device, stream).data_ptr(), nbytes
    _tensor("workspace", workspace, (torch.uint8,), 1, device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel()


def attn_decode_paged(q, k_cache, v_cache, page_table, seq_lens, scale: float | None = None, *,
                      k_scale=None, v_scale=None, workspace=None, out=None, stream=None):
    """Attention of one new query token per sequence over its cached positions.

    ``q``: [B, q_heads, d], bf16 or fp16 (the cache's own type unless it is
    e4m3), ``q_heads`` a multiple of the cached heads.  ``scale`` defaults to
    1/sqrt(d).  Returns ``(o, lse)``: o of q's shape and type, lse fp32
    [B, q_heads]; a sequence of length 0 gives zeros and -inf.  ``workspace``:
    a CUDA uint8 tensor of :func:`attn_decode_workspace_bytes` bytes; a table for
    512 positions at most needs none.
    """
    args, device, (_, heads, page_size, d), batch, width, o, lse, stream = _decode_arguments(
        q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, out, stream)
    if workspace is None and width * page_size <= _DIRECT:
        work = None, 0
    else:
        work = _workspace(workspace, (batch, q.shape[1], heads, d), device, stream)
    _call("fat_attn_decode_paged", device, *args, d ** -0.5 if scale is None else scale,
          o.data_ptr(), lse.data_ptr(), *work, _handle(stream, device))
    return o, lse


def kv_block_bounds(k_cache, page_table, seq_lens, bounds, new_tokens: int | None = None, *,
                    k_scale=None, stream=None):
    """Renew the bounds of the blocks (pages) that hold the newest positions.

    ``bounds``: contiguous [num_pages, heads, 2, d] (the cache's type; bf16 or
    fp16 for an e4m3 cache), the elementwise minimum and maximum of each
    block's keys.  The blocks with any of the last ``new_tokens`` positions of
    a sequence are computed anew (all of them if None); the others keep what
    they have.  A page that several sequences share must be filled to the same
    position in each of those (copy it before one of them goes on in it); else
    its bounds are unspecified.  Returns ``bounds``.
    """
    cache, device, kind, (pages, heads, _, d) = _cache(k_cache, None, k_scale, None)
    table = _table(page_table, seq_lens, device)[0]
    _tensor("bounds", bounds, _WIDE if kind == _E4M3 else (k_cache.dtype,), 4, device)
    if bounds.shape != (pages, heads, 2, d) or not bounds.is_contiguous():
        raise ValueError("bounds must be contiguous [num_pages, heads, 2, d]")
    if bounds.requires_grad:
        _gradient()
    new_tokens = 0x7fffffff if new_tokens is None else int(new_tokens)
    if not 1 <= new_tokens <= 0x7fffffff:
        raise ValueError("new_tokens must be at least 1")
    _call("fat_kv_block_bounds", device, cache, table, new_tokens, bounds.data_ptr(),
          _WIDE[bounds.dtype], _handle(_given(stream, device), device))
    return bounds


def kv_block_scores(q, bounds, page_table, seq_lens, page_size: int, *, out=None, stream=None):
    """Score every block of every sequence for :func:`attn_decode_sparse`.

    ``q``: [B, q_heads, d] of the type of ``bounds`` (see
    :func:`kv_block_bounds`).  Returns fp32 [B, heads, width]: the largest, over
    the query heads that share a cached head, of an upper bound on q . k over
    the block's keys; -inf behind a sequence's last block.
    """
    _tensor("bounds", bounds, _WIDE, 4)
    device = bounds.device
    pages, heads, two, d = bounds.shape
    if two != 2 or not bounds.is_contiguous():
        raise ValueError("bounds must be contiguous [num_pages, heads, 2, d]")
    table, batch, width = _table(page_table, seq_lens, device)
    query = _query(q, batch, heads, d, device)
    if q.dtype is not bounds.dtype:
        raise ValueError("q and bounds must have the same type")
    if not 1 <= page_size <= _MOST:
        raise ValueError("page_size must be a power of two, 16 to 1024")
    if bounds.requires_grad:
        _gradient()
    stream = _given(stream, device)
    if out is None:
        out = _empty((batch, heads, width), torch.float32, device, stream)
    else:
        _output("out", out, (batch, heads, width), torch.float32, device)
    _call("fat_kv_block_scores", device, *query, bounds.data_ptr(), pages, heads, int(page_size),
          d, table, out.data_ptr(), _handle(stream, device))
    return out


def attn_decode_sparse(q, k_cache, v_cache, page_table, seq_lens, scores, num_blocks: int,
                       scale: float | None = None, *, first_blocks: int = 0,
                       last_blocks: int = 1, k_scale=None, v_scale=None, workspace=None,
                       out=None, stream=None):
    """Attention of one new query token per sequence over its best blocks.

    ``scores``: contiguous fp32 [B, heads, width], from :func:`kv_block_scores`
    or any other source.  Each (sequence, cached head) takes the
    ``num_blocks`` blocks (pages) with the highest scores, all if it has no
    more: the last ``last_blocks`` and the first ``first_blocks`` ahead of all
    others (together at most ``num_blocks``), NaN as the highest score, the
    lower index of equal ones.  Returns ``(o, lse, blocks)``: o and lse as in
    :func:`attn_decode_paged`, over the chosen blocks; blocks int32 [B, heads,
    num_blocks], the choice in rising order, then -1.  ``out``: optional
    ``(o, lse, blocks)``.
    """
    args, device, (_, heads, _, d), batch, width, o, lse, stream = _decode_arguments(
        q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, out, stream)
    num_blocks = int(num_blocks)
    if not 1 <= num_blocks <= _MOST or first_blocks < 0 or last_blocks < 0 or \
            first_blocks + last_blocks > num_blocks:
        raise ValueError("num_blocks must be 1 to 2^30 and at least first_blocks + last_blocks")
    _output("scores", scores, (batch, heads, width), torch.float32, device)
    shape = (batch, heads, num_blocks)
    if out is None:
        blocks = _empty(shape, torch.int32, device, stream)
    else:
        blocks = _output("blocks", out[2], shape, torch.int32, device)
    work = _workspace(workspace, (batch, q.shape[1], heads, d, num_blocks), device, stream)
    _call("fat_attn_decode_sparse", device, *args, scores.data_ptr(), num_blocks,
          int(first_blocks), int(last_blocks), d ** -0.5 if scale is None else scale,
          o.data_ptr(), lse.data_ptr(), blocks.data_ptr(), *work, _handle(stream, device))
    return o, lse, blocks
