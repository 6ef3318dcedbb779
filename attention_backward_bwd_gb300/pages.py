"""Binding of the operators on pages that sequences share (include/attn_cache8.h): forking, freeing
and room for new tokens, and the copy of pages.

Argument marshalling only, like cache.py, whose conventions hold here too.
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from .binding import AttnError, _new, _side, lib
from .cache import _DTYPES, _I32, _PAGED, _call, _int32, _ints, _pack, _rows, _workspace
from .cache8 import _FACTORS, _KINDS, _pack_factors


@functools.lru_cache(maxsize=256)
def fork_workspace_size(rows: int, max_pages: int, num_pages: int) -> int:
    return int(lib().attn_cache_fork_workspace_size(rows, max_pages, num_pages))


def _table(name, t, index, shape=None):
    if t.get_device() != index or t.dtype is not _I32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or \
            (shape is not None and t.shape != shape):
        raise AttnError(-9, f"{name} must be an int32 tensor {'[rows, pages]' if shape is None else tuple(shape)} on "
                            f"cuda:{index} with contiguous rows, got {t.dtype} {tuple(t.shape)} on {t.device}")


def attn_cache_fork(block_table, seqlens, refs, page_size: int, parents=None, room=0, share: bool = True,
                    table_out=None, seqlens_out=None, refs_out=None, copies=None, counts=None, workspace=None,
                    stream=None):
    """Forks, reorders and frees sequences and finds pages for new tokens: returns (table, seqlens,
    refs, copies, counts), the first three in place unless ``*_out`` are given.

    ``refs`` (int32 [pages]): how many entries of ``block_table`` (int32 [B, pages a sequence]; -1:
    none) name each page.  Row b becomes that of ``parents[b]`` (int32 [B]; None: its own; negative:
    none, the row is freed).  The first row of a parent goes on with its pages; the others share the
    full ones and get a fresh page for the rest (``share=False``: for all), listed in ``copies``
    (int32 [B, 2], or [B * pages a sequence, 2] without sharing: source, fresh page).  Then every
    row gets fresh pages for ``room`` more slots (an int, or int32 [B]).  Fresh pages are the lowest
    unreferenced ones; ``counts`` (int32 [2]): the copies listed, the pages still free.  Run
    ``attn_cache_copy(..., copies, counts)`` for every cache of the table before the next append.
    """
    if not block_table.is_cuda:
        raise AttnError(-9, f"block_table must be a CUDA tensor, got {block_table.device}")
    index = block_table.get_device()
    _table("block_table", block_table, index)
    rows, width = block_table.shape
    if refs.dim() != 1:
        raise AttnError(-9, f"refs must be a 1-D int32 tensor, got {tuple(refs.shape)}")
    pages = refs.shape[0]
    table_out = block_table if table_out is None else table_out
    seqlens_out = seqlens if seqlens_out is None else seqlens_out
    refs_out = refs if refs_out is None else refs_out
    _table("table_out", table_out, index, block_table.shape)
    lens, lens_out = _ints("seqlens", seqlens, index, rows), _ints("seqlens_out", seqlens_out, index, rows)
    r, r_out = _ints("refs", refs, index, pages), _ints("refs_out", refs_out, index, pages)
    who = _ints("parents", parents, index, rows)
    more, more_all = None, 0
    if isinstance(room, torch.Tensor):
        more = _ints("room", room, index, rows)
    else:
        more_all = _int32("room", room)
    page_size = _int32("page_size", page_size)
    if rows and pages and width and rows * width >= 2**31:
        raise AttnError(-2, "the table must have less than 2^31 entries")
    side = _side(stream, index)
    most = rows if share else rows * width
    if copies is None:
        copies = _new(side, torch.empty, (most, 2), dtype=_I32, device=block_table.device)
    elif copies.get_device() != index or copies.dtype is not _I32 or copies.dim() != 2 or copies.shape[1] != 2 or \
            copies.shape[0] < most or not copies.is_contiguous():
        raise AttnError(-9, f"copies must be a contiguous int32 tensor [>= {most}, 2] on cuda:{index}, got "
                            f"{copies.dtype} {tuple(copies.shape)} on {copies.device}")
    if counts is None:
        counts = _new(side, torch.empty, 2, dtype=_I32, device=block_table.device)
    n = _ints("counts", counts, index, 2)
    ws, size, _held = _workspace(workspace, fork_workspace_size(rows, width, pages), block_table, index, side)
    _call(lib().attn_cache_fork, index, stream, block_table.data_ptr(), block_table.stride(0), table_out.data_ptr(),
          table_out.stride(0), lens, lens_out, r, r_out, pages, rows, width, page_size, who, more, more_all,
          1 if share else 0, copies.data_ptr(), n, ws, size)
    return table_out, seqlens_out, refs_out, copies, counts


def attn_cache_copy(k_cache, v_cache, pairs, counts=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Copies pages of a cache in place: page ``pairs[i, 1]`` becomes page ``pairs[i, 0]`` (int32 [N, 2]).

    ``counts`` (int32, its first entry): how many of the pairs hold, e.g. attn_cache_fork's.  ``k_cache``,
    ``v_cache``: [pages, page_size, H_k, D] in 16 or in 8 bits, the latter with their ``k_scale`` and
    ``v_scale``.  A target must be neither a source nor another target."""
    dtype = k_cache.dtype
    if not k_cache.is_cuda:
        raise AttnError(-9, f"k_cache must be a CUDA tensor, got {k_cache.device}")
    index = k_cache.get_device()
    eight = dtype in _KINDS
    if not eight and dtype not in _DTYPES:
        raise AttnError(-1, f"k_cache must be float16, bfloat16, float8_e4m3fn or int8, got {dtype}")
    ks, vs = _rows("k_cache", k_cache, index, dtype, 4), _rows("v_cache", v_cache, index, dtype, 4)
    if v_cache.shape != k_cache.shape:
        raise AttnError(-2, f"v_cache has shape {tuple(v_cache.shape)}, k_cache {tuple(k_cache.shape)}")
    if eight != (k_scale is not None) or eight != (v_scale is not None):
        raise AttnError(-9, "k_scale and v_scale belong to a cache in 8 bits")
    if pairs.get_device() != index or pairs.dtype is not _I32 or pairs.dim() != 2 or pairs.shape[1] != 2 or \
            not pairs.is_contiguous():
        raise AttnError(-9, f"pairs must be a contiguous int32 tensor [N, 2] on cuda:{index}, got "
                            f"{pairs.dtype} {tuple(pairs.shape)} on {pairs.device}")
    if counts is not None and (counts.get_device() != index or counts.dtype is not _I32 or counts.numel() < 1):
        raise AttnError(-9, f"counts must be an int32 tensor on cuda:{index}, got {counts.dtype} on {counts.device}")
    pages, size, heads, dim = k_cache.shape
    number = _int32("the pairs' number", pairs.shape[0])
    cache = _pack(_PAGED, k_cache.data_ptr(), ks[0], ks[1], ks[2], v_cache.data_ptr(), vs[0], vs[1], vs[2], 0, 0, pages,
                  size, 0)
    cache += _pack_factors(k_cache, k_scale, v_scale, index, _KINDS[dtype]) if eight else _FACTORS.pack(*[0] * 10)
    _call(lib().attn_cache_copy, index, stream, cache, 1 if eight else 2, heads, dim, pairs.data_ptr(),
          None if counts is None else counts.data_ptr(), number)
