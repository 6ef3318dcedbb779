"""Binding of the cache in 8 bits (include/attn_cache8.h): its append, its read-back and attention
of one new token over it.

Argument marshalling only, like cache.py, whose conventions hold here too.  A cache is four
tensors: codes ``k_cache`` and ``v_cache`` [pages, page_size, H_k, D], float8_e4m3fn or int8, any
strides that are multiples of 16 with a contiguous D (a multiple of 16), and ``k_scale`` and
``v_scale``, fp32 [pages, page_size / block, H_k], any positive strides: a factor for each ``block``
neighbouring slots of a page and head.  A cache starts out with any factors and codes.
"""
from __future__ import annotations

import struct
from typing import Optional, Sequence, Tuple

import torch

from .binding import AttnError, _new, _side, lib
from .cache import (_DTYPES, _F32, _OPTS, _PAGED, _batch, _cache, _call, _first, _int32, _ints, _output, _pack, _rotary,
                    _rows, _tensor, _workspace, decode_workspace_size)

_KINDS = {torch.float8_e4m3fn: 0, torch.int8: 1}
# attn_paged_kv8 behind its attn_paged_kv
_FACTORS = struct.Struct("@PPqqqqqqii")


def _factors(name, t, index, shape, page_size):
    s = t.shape
    if t.get_device() != index or t.dtype is not _F32 or len(s) != 3 or s[0] != shape[0] or s[2] != shape[2] or \
            s[1] < 1 or page_size % s[1] != 0:
        raise AttnError(-9, f"{name} must be a float32 tensor [{shape[0]}, blocks of a page of {page_size}, {shape[2]}] "
                            f"on cuda:{index}, got {t.dtype} {tuple(s)} on {t.device}")
    return t.stride()


def _cache8(k_cache, v_cache, k_scale, v_scale, table, index, batch):
    """(attn_paged_kv8, H_k, D, slots of a sequence)."""
    dtype = k_cache.dtype
    kind = _KINDS.get(dtype)
    if kind is None:
        raise AttnError(-1, f"k_cache must be float8_e4m3fn or int8, got {dtype}")
    kv, heads, dim, slots = _cache(k_cache, v_cache, table, index, dtype, batch)
    return kv + _pack_factors(k_cache, k_scale, v_scale, index, kind), heads, dim, slots


def _pack_factors(k_cache, k_scale, v_scale, index, kind) -> bytes:
    shape = k_cache.shape
    size = shape[1]
    ks = _factors("k_scale", k_scale, index, shape, size)
    vs = _factors("v_scale", v_scale, index, shape, size)
    if v_scale.shape != k_scale.shape:
        raise AttnError(-2, f"v_scale has shape {tuple(v_scale.shape)}, k_scale {tuple(k_scale.shape)}")
    return _pack(_FACTORS, k_scale.data_ptr(), v_scale.data_ptr(), *ks, *vs, size // k_scale.shape[1], kind)


def attn_cache_append8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, cu_seqlens=None, q=None,
                       positions=None, inv_freq=None, sections: Optional[Sequence[int]] = None,
                       interleaved: bool = False, out_q=None, stream=None) -> Optional[torch.Tensor]:
    """Stores new keys and values in a paged cache of 8 bits; returns q rotated (None without q).

    As attn_cache_append, with k and v rounded to codes on their way.  The factor of a block of
    slots and head becomes the smallest power of two s (2^-60 .. 2^60) with |x| <= 448 s (int8:
    127 s) for its new values, but not less than that of its earlier slots (below ``seqlens``),
    whose codes are rounded again where it grows."""
    index, dtype, dt = _first(k, "k")
    sk, sv = _rows("k", k, index, dtype, 3), _rows("v", v, index, dtype, 3)
    tokens, hk, d = k.shape
    if v.shape != k.shape:
        raise AttnError(-2, f"v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
    batch = _batch(seqlens)
    _int32("the tokens' number", tokens)
    lens = _ints("seqlens", seqlens, index, batch)
    cache, heads, dim, _ = _cache8(k_cache, v_cache, k_scale, v_scale, block_table, index, batch)
    if heads != hk or dim != d:
        raise AttnError(-2, f"k {tuple(k.shape)} does not fit a cache {tuple(k_cache.shape)}")
    cu = _ints("cu_seqlens", cu_seqlens, index, batch + 1)
    if cu is None and tokens != batch:
        raise AttnError(-9, f"without cu_seqlens there is one token a sequence: {tokens} tokens, "
                            f"{batch} sequences")
    if (positions is None) != (inv_freq is None):
        raise AttnError(-9, "positions and inv_freq go together")
    rot = None if positions is None else \
        _rotary(positions, inv_freq, sections, interleaved, False, index, (tokens,), tokens)
    side = _side(stream, index)
    q_arg = oq_arg = None
    hq = hk
    if q is not None:
        if rot is None:
            raise AttnError(-9, "q is only taken to be rotated: give positions and inv_freq, or no q")
        sq = _rows("q", q, index, dtype, 3)
        hq = q.shape[1]
        if q.shape != (tokens, hq, d):
            raise AttnError(-2, f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree on tokens or D")
        out_q, so = _output("out_q", out_q, q, sq, index, dtype, side)
        q_arg = _tensor(q.data_ptr(), 0, sq[0], sq[1])
        oq_arg = _tensor(out_q.data_ptr(), 0, so[0], so[1])
    elif out_q is not None:
        raise AttnError(-9, "out_q without q")
    if tokens == 0:
        return out_q
    _call(lib().attn_cache_append8, index, stream, q_arg, oq_arg,
          _tensor(k.data_ptr(), 0, sk[0], sk[1]), _tensor(v.data_ptr(), 0, sv[0], sv[1]), dt,
          tokens, batch, hq, hk, d, cache, lens, cu, rot)
    return out_q


def attn_cache_load8(k_cache, v_cache, k_scale, v_scale, block_table, starts, cu_seqlens, tokens: int,
                     dtype=torch.bfloat16, out_k=None, out_v=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Reads slots of a cache of 8 bits back: (k, v), packed [tokens, H_k, D] of ``dtype``.

    Row t, the i-th of sequence b by ``cu_seqlens`` (int32 [B + 1]), is slot ``starts[b] + i``
    (int32 [B]); rows from ``cu_seqlens[B]`` on are left as they were.  With ``starts`` 0 it gives
    the keys and values of a prefix, which attn_fwd attends for the next chunk of a prompt;
    with an append's ``seqlens`` and ``cu_seqlens`` what that append stored."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise AttnError(-1, f"dtype must be float16 or bfloat16, got {dtype}")
    if not k_cache.is_cuda:
        raise AttnError(-9, f"k_cache must be a CUDA tensor, got {k_cache.device}")
    index = k_cache.get_device()
    if starts.dim() != 1:
        raise AttnError(-9, f"starts must be a 1-D int32 tensor, got {tuple(starts.shape)}")
    batch = starts.shape[0]
    tokens = _int32("tokens", tokens)
    if tokens < 0:
        raise AttnError(-2, f"tokens must be >= 0, got {tokens}")
    at = _ints("starts", starts, index, batch)
    cu = _ints("cu_seqlens", cu_seqlens, index, batch + 1)
    if cu is None:
        raise AttnError(-9, "cu_seqlens must be given")
    cache, hk, d, _ = _cache8(k_cache, v_cache, k_scale, v_scale, block_table, index, batch)
    side = _side(stream, index)
    both = []
    for name, out in (("out_k", out_k), ("out_v", out_v)):
        if out is None:
            out = _new(side, torch.empty, (tokens, hk, d), dtype=dtype, device=k_cache.device)
        elif out.shape != (tokens, hk, d):
            raise AttnError(-2, f"{name} has shape {tuple(out.shape)}, {(tokens, hk, d)} was expected")
        both.append((out, _rows(name, out, index, dtype, 3)))
    (out_k, sk), (out_v, sv) = both
    if tokens == 0 or batch == 0:
        return out_k, out_v
    _call(lib().attn_cache_load8, index, stream, _tensor(out_k.data_ptr(), 0, sk[0], sk[1]),
          _tensor(out_v.data_ptr(), 0, sv[0], sv[1]), dt, tokens, batch, hk, d, cache, at, cu)
    return out_k, out_v


def attn_decode8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, max_seqlen: Optional[int] = None,
                 scale: Optional[float] = None, window=None, softcap: float = 0.0, out=None, lse=None,
                 workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of one new token a sequence over a paged cache of 8 bits: (O like q, LSE fp32 [B, H_q]).

    As attn_decode without its ``weights``, on codes and their factors.  ``workspace``: uint8 of at
    least ``decode_workspace_size(...)`` bytes."""
    index, dtype, dt = _first(q, "q")
    sq = _rows("q", q, index, dtype, 3)
    batch, hq, d = q.shape
    cache, hk, dim, slots = _cache8(k_cache, v_cache, k_scale, v_scale, block_table, index, batch)
    if dim != d or hk == 0 or hq % hk != 0:
        raise AttnError(-2, f"q {tuple(q.shape)} does not fit a cache {tuple(k_cache.shape)}")
    lens = _ints("seqlens", seqlens, index, batch)
    max_seqlen = _int32("max_seqlen", slots if max_seqlen is None else max_seqlen)
    side = _side(stream, index)
    out, so = _output("out", out, q, sq, index, dtype, side)
    if lse is None:
        lse = _new(side, torch.empty, (batch, hq), dtype=_F32, device=q.device)
    elif lse.get_device() != index or lse.dtype is not _F32 or lse.shape != (batch, hq) or \
            not lse.is_contiguous():
        raise AttnError(-2, f"lse must be a contiguous float32 tensor {(batch, hq)} on cuda:{index}")
    if batch == 0:
        return out, lse
    ws, size, _held = _workspace(workspace, decode_workspace_size(batch, hq, hk, d, max_seqlen), q, index, side)
    opts = None
    if window is not None or softcap:
        left, right = (-1, -1) if window is None else (int(window[0]), int(window[1]))
        opts = _pack(_OPTS, left, right, float(softcap or 0.0), 0, 0)
    _call(lib().attn_decode8, index, stream, _tensor(q.data_ptr(), sq[0], 0, sq[1]),
          _tensor(out.data_ptr(), so[0], 0, so[1]), lse.data_ptr(), dt, batch, hq, hk, d,
          d ** -0.5 if scale is None else float(scale), cache, lens, max_seqlen, opts, ws, size)
    return out, lse
