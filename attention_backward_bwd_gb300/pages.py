"""Binding of the operators on pages that sequences share (include/attn_cache8.h): forking, freeing
and room for new tokens, and the copy of pages.

Argument marshalling only, in C++ (csrc/native.cpp); cache.py's conventions hold here too.
"""
from __future__ import annotations

import functools

import torch

from .binding import _new, lib
from .cache8 import _is, _on, native


@functools.lru_cache(maxsize=256)
def fork_workspace_size(rows: int, max_pages: int, num_pages: int) -> int:
    return int(lib().attn_cache_fork_workspace_size(rows, max_pages, num_pages))


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
    row gets fresh pages for ``room`` more slots (an int, or int32 [B]).  A row that goes on gets
    copies and fresh pages as well in place of pages that it would write and others hold: after
    ``seqlens`` was lowered (rejected tokens) call this before the next append.  Fresh pages are the lowest
    unreferenced ones; ``counts`` (int32 [2]): the copies listed, the pages still free.  Run
    ``attn_cache_copy(..., copies, counts)`` for every cache of the table before the next append.
    attn_cache_evict writes pages that rows share: fork what is to be evicted with ``share=False`` from
    the start.
    """
    if stream is not None:
        stream, side = _on(stream, block_table)
        if _is(block_table, 2) and _is(refs, 1):
            rows, width = block_table.shape
            make = functools.partial(_new, side, torch.empty, device=block_table.device)
            if copies is None:
                copies = make((rows if share else rows * width, 2), dtype=torch.int32)
            if counts is None:
                counts = make(2, dtype=torch.int32)
            if workspace is None:
                workspace = make(max(fork_workspace_size(rows, width, refs.shape[0]), 256), dtype=torch.uint8)
    return native().fork(block_table, seqlens, refs, page_size, parents, room, share, table_out, seqlens_out, refs_out,
                         copies, counts, workspace, stream)


def attn_cache_copy(k_cache, v_cache, pairs, counts=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Copies pages of a cache in place: page ``pairs[i, 1]`` becomes page ``pairs[i, 0]`` (int32 [N, 2]).

    ``counts`` (int32, its first entry): how many of the pairs hold, e.g. attn_cache_fork's.  ``k_cache``,
    ``v_cache``: [pages, page_size, H_k, D] in 16 or in 8 bits, the latter with their ``k_scale`` and
    ``v_scale``.  A target must be neither a source nor another target."""
    if stream is not None:
        stream, _ = _on(stream, k_cache)
    native().copy(k_cache, v_cache, pairs, counts, k_scale, v_scale, stream)
