"""Binding of the cache in 8 bits (include/attn_cache8.h): its append, its read-back and attention
of one new token over it.

Argument marshalling only, in C++ (csrc/native.cpp); cache.py's conventions hold here too.  A cache is four
tensors: codes ``k_cache`` and ``v_cache`` [pages, page_size, H_k, D], float8_e4m3fn or int8, any
strides that are multiples of 16 with a contiguous D (a multiple of 16), and ``k_scale`` and
``v_scale``, fp32 [pages, page_size / block, H_k], any positive strides: a factor for each ``block``
neighbouring slots of a page and head.  A cache starts out with any factors and codes.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

import torch

from .binding import AttnError, _new, _side, lib
from .cache import _DTYPES, decode_workspace_size

_ENTRIES = ("attn_cache_append8", "attn_cache_load8", "attn_decode8", "attn_decode_workspace_size", "attn_cache_fork",
            "attn_cache_fork_workspace_size", "attn_cache_copy", "attn_last_error")
_native = None


def native():
    """The marshalling module, with the library's entry points (loaded once).  Raises if it has not been built."""
    global _native
    if _native is None:
        library = lib()
        from .build import NATIVE
        if not os.path.exists(NATIVE):
            raise ImportError(f"{NATIVE} is missing: build it with `python -c 'import __graft_entry__ as g; "
                              f"g.build()'`, with a torch that has CUDA.  There is no fallback implementation.")
        from . import _native as module
        module.bind(AttnError, *(ctypes.cast(getattr(library, n), ctypes.c_void_p).value for n in _ENTRIES))
        _native = module
    return _native


def _on(stream, tensor):
    """(stream handle, stream) of an explicit ``stream``: what a call allocates belongs to it."""
    side = _side(stream, tensor.device.index) if isinstance(tensor, torch.Tensor) and tensor.is_cuda else None
    return (stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)), side


def _is(tensor, dims):
    """Whether sizes can be taken from it (the call refuses what is none, as without ``stream``)."""
    return isinstance(tensor, torch.Tensor) and tensor.dim() == dims


def attn_cache_append8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, cu_seqlens=None, q=None,
                       positions=None, inv_freq=None, sections: Optional[Sequence[int]] = None,
                       interleaved: bool = False, out_q=None, stream=None) -> Optional[torch.Tensor]:
    """Stores new keys and values in a paged cache of 8 bits; returns q rotated (None without q).

    As attn_cache_append, with k and v rounded to codes on their way.  The factor of a block of
    slots and head becomes the smallest power of two s (2^-60 .. 2^60) with |x| <= 448 s (int8:
    127 s) for its new values, but not less than that of its earlier slots (below ``seqlens``),
    whose codes are rounded again where it grows."""
    if stream is not None:
        stream, side = _on(stream, k)
        if _is(q, 3) and out_q is None:
            out_q = _new(side, torch.empty_like, q)
    return native().append8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, cu_seqlens, q, positions,
                            inv_freq, sections, interleaved, out_q, stream)


def attn_cache_load8(k_cache, v_cache, k_scale, v_scale, block_table, starts, cu_seqlens, tokens: int,
                     dtype=torch.bfloat16, out_k=None, out_v=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Reads slots of a cache of 8 bits back: (k, v), packed [tokens, H_k, D] of ``dtype``.

    Row t, the i-th of sequence b by ``cu_seqlens`` (int32 [B + 1]), is slot ``starts[b] + i``
    (int32 [B]); rows from ``cu_seqlens[B]`` on are left as they were.  With ``starts`` 0 it gives
    the keys and values of a prefix, which attn_fwd attends for the next chunk of a prompt;
    with an append's ``seqlens`` and ``cu_seqlens`` what that append stored."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise AttnError(-1, f"dtype must be float16 or bfloat16, got {dtype}")
    if stream is not None:
        stream, side = _on(stream, k_cache)
        if _is(k_cache, 4):
            like = (max(0, tokens), *k_cache.shape[2:])
            out_k, out_v = (_new(side, torch.empty, like, dtype=dtype, device=k_cache.device) if x is None else x
                            for x in (out_k, out_v))
    return native().load8(k_cache, v_cache, k_scale, v_scale, block_table, starts, cu_seqlens, tokens, out_k, out_v,
                          code, stream)


def attn_decode8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, max_seqlen: Optional[int] = None,
                 scale: Optional[float] = None, window=None, softcap: float = 0.0, out=None, lse=None,
                 workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of one new token a sequence over a paged cache of 8 bits: (O like q, LSE fp32 [B, H_q]).

    As attn_decode without its ``weights``, on codes and their factors.  ``workspace``: uint8 of at
    least ``decode_workspace_size(...)`` bytes."""
    if stream is not None:
        stream, side = _on(stream, q)
        fits = _is(q, 3) and _is(k_cache, 4) and _is(block_table, 2)
        if out is None and fits:
            out = _new(side, torch.empty_like, q)
        if lse is None and fits:
            lse = _new(side, torch.empty, q.shape[:2], dtype=torch.float32, device=q.device)
        if workspace is None and fits:
            most = block_table.shape[1] * k_cache.shape[1] if max_seqlen is None else max_seqlen
            need = decode_workspace_size(*q.shape[:2], k_cache.shape[2], q.shape[2], most)
            workspace = _new(side, torch.empty, max(need, 256), dtype=torch.uint8, device=q.device)
    return native().decode8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, max_seqlen, scale, window,
                            softcap, out, lse, workspace, stream)
