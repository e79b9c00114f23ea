"""A step of drafted tokens over the paged cache of :mod:`.paged`: the binding of
``fat_kv_append``, ``fat_attn_tree_paged`` and ``fat_kv_keep`` of
``include/fat_attn.h``.

Several tokens are drafted for every sequence, stored in its cache with their
keys rotated (:func:`kv_cache_append`), judged by one pass of attention in which
each sees its sequence's context and its own ancestors (:func:`attn_tree_paged`),
and the accepted ones are moved right behind the context (:func:`kv_cache_keep`).
:func:`kv_cache_append` is as well the way in for prompts and single tokens.

What :mod:`.paged` says of caches, tables, streams, workspaces, graphs and
gradients holds here too.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _empty, _given, load_library
from .paged import (
    _E4M3, _F, _I, _L, _P, _WIDE, _Z, _cache, _call, _gradient, _handle, _output, _table,
    _tensor, _tokens,
)

_AXES = 4  # FAT_ROTATION_AXES
_TREE = 64  # FAT_TREE_TOKENS


class FatRotation(ctypes.Structure):
    """Mirror of ``fat_rotation`` in include/fat_attn.h (same field order)."""
    _fields_ = [("cos_sin", _P), ("rows", _L), ("row_stride", _L), ("positions", _P),
                ("axis_stride", _L), ("token_stride", _L), ("dim", _I), ("axes", _I),
                ("sections", _I * _AXES), ("interleaved", _I)]


_pack_rotation = struct.Struct("@PqqPqqii4ii4x").pack


def declare(lib) -> None:
    """Argument and result types of the entry points used here."""
    tree = [_P, _P, _P, _I, _L, _L, _L, _I, _I, _P, _L, _P, _I, _I, _F, _P, _P, _P, _Z]
    for name, args, result in (
            ("fat_kv_append", [_P, _P, _P, _L, _L, _I, _P, _P, _I, _L, _L, _L, _L, _P, _I, _P, _P],
             _I),
            ("fat_kv_keep", [_P, _P, _P, _L, _I, _P, _P], _I),
            ("fat_attn_tree_paged", [*tree, _P], _I),
            ("fat_attn_tree_paged_ex", [*tree, ctypes.c_ulonglong, _P], _I),
            ("fat_attn_tree_workspace_bytes", [_I, _I, _I, _I, _I], _Z)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, result


def _rotation(cos_sin, positions, sections, interleaved, tokens, d, device):
    """The checked rotation as a packed struct."""
    _tensor("cos_sin", cos_sin, (torch.float32,), 2, device)
    rows, dim = cos_sin.shape
    stride, step = cos_sin.stride()
    if cos_sin.requires_grad:
        _gradient()
    if dim % 16 or not 16 <= dim <= d or rows < 1:
        raise ValueError(f"cos_sin must be [positions, a multiple of 16 up to {d}], "
                         f"not {list(cos_sin.shape)}")
    if step != 1:
        raise ValueError("the rows of cos_sin must be contiguous")
    if sections is None:
        axes, parts = 1, (dim // 2,)
        _tensor("positions", positions, (torch.int64,), 1, device)
        shape, along, step = (tokens,), 0, positions.stride(0)
    else:
        parts = tuple(int(n) for n in sections)
        axes = len(parts)
        if not 1 <= axes <= _AXES or min(parts) < 0 or sum(parts) != dim // 2:
            raise ValueError(f"sections must be up to {_AXES} counts of pairs that add up to "
                             f"{dim // 2}, not {parts}")
        _tensor("positions", positions, (torch.int64,), 2, device)
        shape, (along, step) = (axes, tokens), positions.stride()
    if positions.shape != shape:
        raise ValueError(f"positions must be {list(shape)}, not {list(positions.shape)}")
    return _pack_rotation(cos_sin.data_ptr(), rows, stride if rows > 1 else max(stride, dim),
                          positions.data_ptr(), along if axes > 1 else 0, step, dim, axes, *parts,
                          *(0,) * (_AXES - axes), 1 if interleaved else 0)


def kv_cache_append(q, k, v, k_cache, v_cache, slots, positions, cos_sin, *, sections=None,
                    interleaved: bool = False, k_scale=None, v_scale=None, out=None, stream=None):
    """Store new tokens with their keys rotated, and rotate their queries.

    ``k, v, slots, k_scale, v_scale`` as in :func:`.kv_cache_write`; ``q``: [T,
    q_heads, d] of k's type, or None.  ``cos_sin``: fp32 [P, n], the cosines of
    the n / 2 rotated pairs at each position, then their sines; n, a multiple of
    16 up to d, says how many leading elements of a row are rotated, in pairs
    (i, i + n / 2) or with ``interleaved`` (2 i, 2 i + 1).  ``positions``: int64
    [T]; or with ``sections``, the counts of pairs that belong to each of up to
    four axes (time, height and width, say), int64 [axes, T].  A key is rounded
    once, to the cache's type.  The slots of one call must differ.  Tokens with a
    negative slot are not stored, their queries are rotated all the same.  A
    position outside the table cannot be refused here: nothing of that token is
    stored or given out, and :func:`check_device_error` returns ``FAT_ERR_INDEX``.

    Returns the rotated queries, contiguous [T, q_heads, d] (None without q);
    ``out``: a tensor for them, which may be a contiguous q itself.
    """
    cache, device, kind, (_, heads, _, d) = _cache(k_cache, v_cache, k_scale, v_scale, True)
    _tensor("slots", slots, (torch.int64,), 1, device)
    tokens = slots.shape[0]
    k_strides = _tokens("k", k, (tokens, heads, d), _WIDE, device)
    v_strides = _tokens("v", v, (tokens, heads, d), (k.dtype,), device)
    if kind != _E4M3 and k.dtype != k_cache.dtype:
        raise ValueError(f"a {k_cache.dtype} cache takes {k_cache.dtype} tokens, not {k.dtype}")
    if k.requires_grad or v.requires_grad:
        _gradient()
    if not slots.is_contiguous():
        raise ValueError("slots must be contiguous")
    stream = _given(stream, device)
    q_args, q_out = (None, 0, 0, 0), None
    if q is not None:
        _tensor("q", q, (k.dtype,), 3, device)
        shape = (tokens, q.shape[1], d)
        if q.shape[1] < 1:
            raise ValueError("q must have heads")
        q_strides = _tokens("q", q, shape, (k.dtype,), device)
        if q.requires_grad:
            _gradient()
        q_args = (q.data_ptr(), *q_strides, shape[1])
        q_out = _empty(shape, q.dtype, device, stream) if out is None \
            else _output("out", out, shape, q.dtype, device)
    elif out is not None:
        raise ValueError("out goes with q")
    rotation = _rotation(cos_sin, positions, sections, interleaved, tokens, d, device)
    if not tokens:
        return q_out
    if tokens > 0x7fffffff:
        raise ValueError("more than 2^31 - 1 tokens in one call")
    _call("fat_kv_append", device, cache, rotation, *q_args, k.data_ptr(), v.data_ptr(),
          _WIDE[k.dtype], *k_strides, *v_strides, slots.data_ptr(), tokens,
          None if q_out is None else q_out.data_ptr(), _handle(stream, device))
    return q_out


def tree_mask(parents):
    """The masks of :func:`attn_tree_paged` from the drafted tokens' parents.

    ``parents``: integers [..., T], T up to 64: the index of each token's parent,
    an earlier drafted token, or -1 for a child of the context's last token (what
    is no earlier token counts as -1).  Returns int64 [..., T]: each token's
    ancestors and itself as bits.  Plain torch operations on the parents' device,
    T steps: for a tree that many steps use.
    """
    tokens = parents.shape[-1] if parents.dim() else 0
    if parents.is_floating_point() or not 1 <= tokens <= _TREE:
        raise ValueError(f"parents must be integers [..., 1 to {_TREE}]")
    masks = torch.zeros(parents.shape, dtype=torch.int64, device=parents.device)
    for t in range(tokens):
        p = parents[..., t].long()
        up = masks.gather(-1, p.clamp(0, tokens - 1)[..., None])[..., 0]
        own = (1 << t) - (1 << 64 if t == 63 else 0)
        masks[..., t] = torch.where((p >= 0) & (p < t), up, torch.zeros_like(up)) | own
    return masks


@functools.lru_cache(maxsize=256)
def attn_tree_workspace_bytes(batch: int, tokens: int, q_heads: int, kv_heads: int,
                              d: int) -> int:
    """Workspace size of :func:`attn_tree_paged` (0 for invalid arguments)."""
    return load_library().fat_attn_tree_workspace_bytes(batch, tokens, q_heads, kv_heads, d)


def attn_tree_paged(q, k_cache, v_cache, page_table, seq_lens, tree, scale: float | None = None, *,
                    draft_lens=None, window: int | None = None, sinks: int = 0, k_scale=None,
                    v_scale=None, workspace=None, out=None, stream=None,
                    wait_timeout_ns: int = 0):
    """Attention of up to 64 drafted tokens per sequence over its cached positions.

    The drafted tokens' keys and values are in the cache already, as the last
    positions of each sequence: ``seq_lens`` counts them, all T of ``q`` [B, T,
    q_heads, d], or the first ``draft_lens`` (int32 [B]) of them where fewer were
    drafted.  A token sees its sequence's context, the positions ahead of the
    drafted ones, and the drafted tokens whose bits are set in its mask:
    ``tree``, int64 [B, T], or [T] for all (see :func:`tree_mask`; a chain of
    tokens has the masks 1, 3, 7, ...).  With ``window`` (at least T) a token
    sees only the last ``window`` positions, counted along its own path, and the
    first ``sinks`` ones, as in :func:`.attn_decode_window`.

    ``q``: bf16 or fp16 (the cache's own type unless it is e4m3), a view of rows
    that lie apart (one that repeats heads or tokens is refused with
    ``FAT_ERR_UNSUPPORTED``); ``scale`` defaults to 1/sqrt(d).  Weights are
    rounded to bf16 for a bf16 cache and to fp16 for the others before they meet
    the values (:func:`.attn_decode_paged` carries a second 16-bit term of them);
    values times the positions that a row sees have to stay below 2^120 over a bf16
    cache, 2^113 over an e4m3 one.  Returns ``(o, lse)``: o contiguous of q's shape and
    type, lse fp32 [B, T, q_heads]; rows that see nothing and rows from
    ``draft_lens`` on are zeros and -inf.  ``workspace``: a CUDA uint8 tensor of
    :func:`attn_tree_workspace_bytes` bytes.  ``wait_timeout_ns``: a limit for each
    wait inside the kernel instead of 4 s, for tests; where one runs out the results
    are unspecified and :func:`check_device_error` returns ``FAT_ERR_DEVICE_TIMEOUT``.
    """
    cache, device, kind, (_, heads, _, d) = _cache(k_cache, v_cache, k_scale, v_scale)
    table, batch, _ = _table(page_table, seq_lens, device)
    _tensor("q", q, _WIDE, 4, device)
    _, tokens, q_heads, width = q.shape
    if q.requires_grad:
        _gradient()
    if q.shape[0] != batch or width != d or not 1 <= tokens <= _TREE or q_heads < 1 or \
            q_heads % heads:
        raise ValueError(f"q must be [{batch}, 1 to {_TREE}, a multiple of {heads}, {d}], "
                         f"not {list(q.shape)}")
    if kind != _E4M3 and q.dtype != k_cache.dtype:
        raise ValueError(f"a {k_cache.dtype} cache takes {k_cache.dtype} queries, not {q.dtype}")
    per_batch, per_token, per_head, step = q.stride()
    if step != 1:
        raise ValueError("the rows of q must be contiguous")
    if not isinstance(tree, torch.Tensor) or tree.dim() not in (1, 2):
        raise ValueError("tree must be an int64 tensor [B, T] or [T]")
    _tensor("tree", tree, (torch.int64,), tree.dim(), device)
    shape = (tokens,) if tree.dim() == 1 else (batch, tokens)
    if tree.shape != shape or (tree.stride(-1) != 1 and tokens > 1):
        raise ValueError(f"tree must be {list(shape)} with contiguous rows")
    tree_stride = tree.stride(0) if tree.dim() == 2 and batch > 1 else 0
    if draft_lens is not None:
        _tensor("draft_lens", draft_lens, (torch.int32,), 1, device)
        if draft_lens.shape[0] != batch or not draft_lens.is_contiguous():
            raise ValueError("draft_lens must be contiguous [B]")
    if window is not None and not tokens <= window <= 0x7fffffff:
        raise ValueError(f"window must be at least the {tokens} drafted tokens, below 2^31")
    if not 0 <= sinks <= 0x7fffffff:
        raise ValueError("sinks must be at least 0, below 2^31")
    if sinks and window is None:
        raise ValueError("sinks go with a window")
    if not 0 <= wait_timeout_ns < 1 << 63:
        raise ValueError("wait_timeout_ns must be at least 0, below 2^63")
    stream = _given(stream, device)
    if out is None:
        o = _empty(q.shape, q.dtype, device, stream)
        lse = _empty((batch, tokens, q_heads), torch.float32, device, stream)
    else:
        o = _output("o", out[0], q.shape, q.dtype, device)
        lse = _output("lse", out[1], (batch, tokens, q_heads), torch.float32, device)
    if workspace is None:
        nbytes = attn_tree_workspace_bytes(batch, tokens, q_heads, heads, d)
        workspace = _empty((nbytes,), torch.uint8, device, stream)
    else:
        _tensor("workspace", workspace, (torch.uint8,), 1, device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _call("fat_attn_tree_paged_ex", device, cache, table, q.data_ptr(), _WIDE[q.dtype],
          per_batch if batch > 1 else 0, per_token if tokens > 1 else 0,
          per_head if q_heads > 1 else 0, q_heads, tokens, tree.data_ptr(), tree_stride,
          None if draft_lens is None else draft_lens.data_ptr(),
          0 if window is None else int(window), int(sinks), d ** -0.5 if scale is None else scale,
          o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
          int(wait_timeout_ns), _handle(stream, device))
    return o, lse


def kv_cache_keep(k_cache, v_cache, page_table, context_lens, path, counts, *, k_scale=None,
                  v_scale=None, stream=None) -> None:
    """Keep the accepted drafted tokens: move their rows right behind the context.

    ``context_lens``: int32 [B], the positions ahead of the drafted tokens;
    ``path``: int32 [B, M], of each sequence the accepted tokens as indexes among
    its drafted ones, rising; ``counts``: int32 [B], how many of them (0 to M).
    The row at position ``context_lens + path[i]`` moves to ``context_lens + i``,
    in every head, keys, values and scales; the sequence then has
    ``context_lens + counts`` positions.  An entry that leads outside the table
    moves nothing, and :func:`check_device_error` returns ``FAT_ERR_INDEX``.
    Pages that are written to must be the sequence's own.  Block bounds are renewed
    by :func:`.kv_block_bounds` as after a write.
    """
    cache, device, kind, _ = _cache(k_cache, v_cache, k_scale, v_scale, True)
    table, batch, _ = _table(page_table, context_lens, device)
    _tensor("path", path, (torch.int32,), 2, device)
    _tensor("counts", counts, (torch.int32,), 1, device)
    if path.shape[0] != batch or counts.shape[0] != batch or not counts.is_contiguous():
        raise ValueError("path must be [B, M] and counts contiguous [B]")
    width = path.shape[1]
    if not width:
        return
    if path.stride(1) != 1 and width > 1:
        raise ValueError("the rows of path must be contiguous")
    _call("fat_kv_keep", device, cache, table, path.data_ptr(),
          path.stride(0) if batch > 1 else 0, width, counts.data_ptr(),
          _handle(_given(stream, device), device))
