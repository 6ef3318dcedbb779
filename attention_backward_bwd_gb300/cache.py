"""Binding of the serving operators (include/attn_cache.h): rotary positions, the
paged key/value cache's append, attention of one new token over it, and eviction.

Argument marshalling only, like binding.py: every step of the computation runs in
the library's CUDA kernels, there is no fallback, and argument errors raise
AttnError before anything is launched.  Lengths, block tables and offsets live on
the device and are checked there; check_device_status() reports what was bad.

The calls run on the device of their tensors, on ``stream`` (default: that device's
current stream).  What a call allocates itself belongs to that stream; the caller orders
``stream`` behind the work that makes its inputs, and its later work behind ``stream``.
"""
from __future__ import annotations

import functools
import struct
from typing import Optional, Sequence, Tuple

import torch

from .binding import ATTN_BF16, ATTN_FP16, AttnError, _new, _side, lib

_DTYPES = {torch.float16: ATTN_FP16, torch.bfloat16: ATTN_BF16}
# attn_tensor, attn_paged_kv, attn_rotary and attn_opts as a C compiler lays them out
_TENSOR = struct.Struct("@Pqqq")
_PAGED = struct.Struct("@PqqqPqqqPqiii4x")
_ROTARY = struct.Struct("@PqPii4iii")
_OPTS = struct.Struct("@iif4xPP")
_tensor = _TENSOR.pack  # pointers and strides always fit
_I32, _F32 = torch.int32, torch.float32
# The current stream as an integer, without a Stream object around it (a call of a few
# microseconds is mostly marshalling).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _fail(rc: int):
    raise AttnError(rc, lib().attn_last_error().decode())


def _pack(form: struct.Struct, *values) -> bytes:
    try:
        return form.pack(*values)
    except struct.error as e:
        raise AttnError(-9, f"an argument does not fit its C type: {e}") from None


def _int32(name, value) -> int:
    """``value`` as an int that a C int holds (ctypes would drop the upper bits)."""
    value = int(value)
    if not -2**31 <= value < 2**31:
        raise AttnError(-9, f"{name} ({value}) does not fit 32 bits")
    return value


def _call(fn, index, stream, *args):
    """Runs fn(*args, stream) with device ``index`` current."""
    raw = _raw_stream(index) if stream is None else \
        stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        _fail(rc)


def _first(t: torch.Tensor, name: str):
    """(device index, dtype, dtype code) that the call's other tensors have to share."""
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise AttnError(-1, f"{name} must be float16 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise AttnError(-9, f"{name} must be a CUDA tensor, got {t.device}")
    return t.get_device(), t.dtype, code


def _rows(name, t, index, dtype, dims):
    """Strides of a tensor of head rows, after its device, dtype, rank and unit stride
    over the head dimension were checked."""
    s = t.stride()
    if t.get_device() != index or t.dtype is not dtype or len(s) != dims or s[-1] != 1:
        if t.get_device() != index:
            raise AttnError(-9, f"{name} must be a CUDA tensor on cuda:{index}, got {t.device}")
        if t.dtype is not dtype:
            raise AttnError(-1, f"{name} has dtype {t.dtype}, {dtype} was expected")
        if len(s) != dims:
            raise AttnError(-2, f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
        if t.numel() > 0:
            raise AttnError(-3, f"{name} must have unit stride over the head dimension")
    return s


def _ints(name, t, index, n):
    """Pointer of a contiguous int32 tensor of n entries (None: none)."""
    if t is None:
        return None
    if t.get_device() != index or t.dtype is not _I32 or t.dim() != 1 or t.shape[0] != n or \
            not t.is_contiguous():
        raise AttnError(-9, f"{name} must be a contiguous int32 tensor [{n}] on cuda:{index}, got "
                            f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _batch(seqlens) -> int:
    if seqlens.dim() != 1:
        raise AttnError(-9, f"seqlens must be a 1-D int32 tensor, got {tuple(seqlens.shape)}")
    return seqlens.shape[0]


def _state(name, t, index, dtype, batch, heads, width):
    """(pointer, entries of a row) of a contiguous [batch, H_k, >= width] tensor of
    per-slot state."""
    s = t.shape
    if t.get_device() != index or t.dtype is not dtype or len(s) != 3 or s[0] != batch or \
            s[1] != heads or s[2] < width or not t.is_contiguous():
        raise AttnError(-9, f"{name} must be a contiguous {dtype} tensor [{batch}, {heads}, >= {width}] "
                            f"on cuda:{index}, got {t.dtype} {tuple(s)} on {t.device}")
    return t.data_ptr(), s[2]


def _cache(k_cache, v_cache, table, index, dtype, batch):
    """(attn_paged_kv, H_k, D, slots of a sequence)."""
    ks = _rows("k_cache", k_cache, index, dtype, 4)
    vs = _rows("v_cache", v_cache, index, dtype, 4)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise AttnError(-2, f"v_cache has shape {tuple(v_cache.shape)}, k_cache {tuple(shape)}")
    pages, size, heads, dim = shape
    if table.get_device() != index or table.dtype is not _I32 or table.dim() != 2 or \
            table.shape[0] != batch or (table.shape[1] > 1 and table.stride(1) != 1):
        raise AttnError(-9, f"block_table must be an int32 tensor [{batch}, pages] on cuda:{index} with "
                            f"contiguous rows, got {table.dtype} {tuple(table.shape)} on {table.device}")
    per = table.shape[1]
    return _pack(_PAGED, k_cache.data_ptr(), ks[0], ks[1], ks[2], v_cache.data_ptr(), vs[0], vs[1], vs[2],
                       table.data_ptr(), table.stride(0), pages, size, per), heads, dim, per * size


def _rotary(positions, inv_freq, sections, interleaved, inverse, index, lead, tokens) -> bytes:
    if inv_freq.get_device() != index or inv_freq.dtype is not _F32 or inv_freq.dim() != 1 or \
            not inv_freq.is_contiguous():
        raise AttnError(-9, f"inv_freq must be a contiguous 1-D float32 tensor on cuda:{index}")
    n = inv_freq.shape[0]
    sec = (n,) if sections is None else tuple(sections)
    axes = len(sec)
    if not 1 <= axes <= 4:
        raise AttnError(-2, f"sections must name 1 to 4 axes, got {axes}")
    shape = positions.shape
    if shape != (axes, *lead) and not (axes == 1 and shape == lead):
        raise AttnError(-2, f"positions must be {(axes, *lead)}, got {tuple(shape)}")
    if positions.get_device() != index or positions.dtype is not _I32 or not positions.is_contiguous():
        raise AttnError(-9, f"positions must be a contiguous int32 tensor on cuda:{index}, got "
                            f"{positions.dtype} on {positions.device}")
    return _pack(_ROTARY, positions.data_ptr(), tokens, inv_freq.data_ptr(), n, axes,
                        *sec, *(0, 0, 0, 0)[axes:], 1 if interleaved else 0, 1 if inverse else 0)


def _stride3(s):
    """Strides of batch, sequence and head of a padded or packed tensor."""
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


def _output(name, out, x, sx, index, dtype, side):
    """(out, its strides): allocated like x, or checked against it."""
    if out is None:
        out = _new(side, torch.empty_like, x)
        return out, out.stride()
    so = _rows(name, out, index, dtype, len(sx))
    if out.shape != x.shape:
        raise AttnError(-2, f"{name} has shape {tuple(out.shape)}, its input {tuple(x.shape)}")
    if out.data_ptr() == x.data_ptr() and so != sx and out.numel() > 0:
        raise AttnError(-9, f"{name} starts where its input does but has other strides")
    return out, so


def attn_rope(q, k, positions, inv_freq, sections: Optional[Sequence[int]] = None,
              interleaved: bool = False, inverse: bool = False, out_q=None, out_k=None,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions: returns q and k ([B, S, H, D] or packed [total, H, D]) rotated.

    Pair i of a head row turns by ``positions[axis(i), token] * inv_freq[i]``;
    the pair is (i, i + n) with n = ``inv_freq.numel()``, or (2i, 2i + 1) when
    ``interleaved``; elements from 2n on are copied.  ``positions``: int32
    [axes, B, S] / [axes, total] (without the first dimension for one axis);
    ``sections``: frequencies of each axis, at most four, in order (default: one axis).
    ``inverse=True`` turns back: on the gradients of the rotated q and k it is
    the backward pass.  ``k`` may be None.  ``out_q`` / ``out_k`` may be the inputs."""
    index, dtype, dt = _first(q, "q")
    shape = q.shape
    dims = len(shape)
    if dims == 3:
        tokens, hq, d = shape
        batch, seqlen, lead = 1, tokens, (tokens,)
    elif dims == 4:
        batch, seqlen, hq, d = shape
        tokens, lead = batch * seqlen, (batch, seqlen)
    else:
        raise AttnError(-2, f"q must be [B, S, H, D] or packed [total, H, D], got {tuple(shape)}")
    _int32("the tokens' number", tokens)
    side = _side(stream, index)
    sq = _rows("q", q, index, dtype, dims)
    out_q, so = _output("out_q", out_q, q, sq, index, dtype, side)
    hk, pk, pok = hq, None, None
    if k is not None:
        sk = _rows("k", k, index, dtype, dims)
        hk = k.shape[-2]
        if k.shape != (*lead, hk, d):
            raise AttnError(-2, f"q {tuple(shape)} and k {tuple(k.shape)} disagree on tokens or D")
        out_k, sok = _output("out_k", out_k, k, sk, index, dtype, side)
        pk, pok = _tensor(k.data_ptr(), *_stride3(sk)), _tensor(out_k.data_ptr(), *_stride3(sok))
    elif out_k is not None:
        raise AttnError(-9, "out_k without k")
    rot = _rotary(positions, inv_freq, sections, interleaved, inverse, index, lead, tokens)
    if tokens == 0:
        return out_q, out_k
    _call(lib().attn_rope, index, stream, _tensor(q.data_ptr(), *_stride3(sq)), pk,
          _tensor(out_q.data_ptr(), *_stride3(so)), pok, dt, batch, seqlen, hq, hk, d, rot)
    return out_q, out_k


def attn_cache_append(k, v, k_cache, v_cache, block_table, seqlens, cu_seqlens=None, q=None,
                      positions=None, inv_freq=None, sections: Optional[Sequence[int]] = None,
                      interleaved: bool = False, out_q=None, slot_positions=None, seen=None,
                      stream=None) -> Optional[torch.Tensor]:
    """Stores new keys and values in the paged cache; returns q rotated (None without q).

    ``k``, ``v``: packed [tokens, H_k, D]; the i-th token of sequence b goes to slot
    ``seqlens[b] + i`` (``cu_seqlens``: int32 [B + 1]; without it one token a
    sequence; tokens from ``cu_seqlens[B]`` on are left out).  ``k_cache``,
    ``v_cache``: [pages, page_size, H_k, D], any strides with a contiguous D;
    ``block_table``: int32 [B, pages a sequence].  With ``positions`` and
    ``inv_freq`` k is rotated on its way (see attn_rope), and so is ``q``
    [tokens, H_q, D] into ``out_q`` (which may be q).  ``slot_positions`` (int32
    [B, H_k, slots], with ``seen`` int32 [B]) receives each new slot's token
    number ``seen[b] + i`` for attn_cache_evict.  ``seqlens`` is not advanced.
    """
    index, dtype, dt = _first(k, "k")
    sk, sv = _rows("k", k, index, dtype, 3), _rows("v", v, index, dtype, 3)
    tokens, hk, d = k.shape
    if v.shape != k.shape:
        raise AttnError(-2, f"v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
    batch = _batch(seqlens)
    _int32("the tokens' number", tokens)
    lens = _ints("seqlens", seqlens, index, batch)
    cache, heads, dim, _ = _cache(k_cache, v_cache, block_table, index, dtype, batch)
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
    sp, width = None, 0
    if slot_positions is not None:
        if seen is None:
            raise AttnError(-9, "slot_positions needs seen")
        sp, width = _state("slot_positions", slot_positions, index, _I32, batch, hk, 1)
    if tokens == 0:
        return out_q
    _call(lib().attn_cache_append, index, stream, q_arg, oq_arg,
          _tensor(k.data_ptr(), 0, sk[0], sk[1]), _tensor(v.data_ptr(), 0, sv[0], sv[1]), dt,
          tokens, batch, hq, hk, d, cache, lens, cu, rot, sp, width, _ints("seen", seen, index, batch))
    return out_q


@functools.lru_cache(maxsize=256)
def decode_workspace_size(batch: int, h_q: int, h_k: int, head_dim: int, max_seqlen: int,
                          weights: bool = False) -> int:
    return int(lib().attn_decode_workspace_size(batch, h_q, h_k, head_dim, _int32("max_seqlen", max_seqlen),
                                                int(weights)))


def alloc_decode_workspace(q, k_cache, max_seqlen: int, weights: bool = False) -> torch.Tensor:
    """Workspace (at least 256 bytes) of attn_decode for queries like ``q`` [B, H_q, D] over ``k_cache``."""
    n = decode_workspace_size(q.shape[0], q.shape[1], k_cache.shape[2], q.shape[2], max_seqlen, weights)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def _workspace(workspace, need, like, index, side):
    """(pointer, bytes, tensor) of the caller's workspace or of a new one (none if none is needed),
    which the caller holds until its call is queued."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _new(side, torch.empty, need, dtype=torch.uint8, device=like.device)
    elif workspace.get_device() != index or workspace.dtype is not torch.uint8 or \
            not workspace.is_contiguous():
        raise AttnError(-9, f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    return workspace.data_ptr(), workspace.numel(), workspace


def attn_decode(q, k_cache, v_cache, block_table, seqlens, max_seqlen: Optional[int] = None,
                scale: Optional[float] = None, window=None, softcap: float = 0.0, out=None, lse=None,
                weights=None, weights_out=None, workspace=None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of one new token a sequence over the paged cache: (O like q, LSE fp32 [B, H_q]).

    ``q``: [B, H_q, D]; ``seqlens``: int32 [B], the cached keys of each sequence,
    the new token's own among them (0: O = 0 and LSE = +inf); ``max_seqlen``: a
    bound on them (default: what the block table can hold).  ``window`` and
    ``softcap`` as in attn_fwd (the query sits at the last slot, so only the left
    side matters).  ``weights`` (fp32 [B, H_k, >= max_seqlen]): each cached key's
    softmax weight, summed over the query heads that share it, is added to it, in
    place or into ``weights_out``.  ``workspace``: uint8 of at least
    ``decode_workspace_size(...)`` bytes, not shared by calls that may overlap."""
    index, dtype, dt = _first(q, "q")
    sq = _rows("q", q, index, dtype, 3)
    batch, hq, d = q.shape
    cache, hk, dim, slots = _cache(k_cache, v_cache, block_table, index, dtype, batch)
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
    w_in = w_out = None
    width = 0
    if weights is not None:
        w_in, width = _state("weights", weights, index, _F32, batch, hk, max_seqlen)
        w_out = w_in
        if weights_out is not None:
            w_out, other = _state("weights_out", weights_out, index, _F32, batch, hk, max_seqlen)
            if other != width:
                raise AttnError(-2, "weights and weights_out must have the same shape")
    elif weights_out is not None:
        raise AttnError(-9, "weights_out without weights")
    if batch == 0:
        return out, lse
    ws, size, _held = _workspace(workspace, decode_workspace_size(batch, hq, hk, d, max_seqlen, w_in is not None),
                                 q, index, side)
    opts = None
    if window is not None or softcap:
        left, right = (-1, -1) if window is None else (int(window[0]), int(window[1]))
        opts = _pack(_OPTS, left, right, float(softcap or 0.0), 0, 0)
    _call(lib().attn_decode, index, stream, _tensor(q.data_ptr(), sq[0], 0, sq[1]),
          _tensor(out.data_ptr(), so[0], 0, so[1]), lse.data_ptr(), dt, batch, hq, hk, d,
          d ** -0.5 if scale is None else float(scale), cache, lens, max_seqlen, opts, w_in, w_out,
          width, ws, size)
    return out, lse


@functools.lru_cache(maxsize=256)
def evict_workspace_size(batch: int, h_k: int, budget: int, max_seqlen: int) -> int:
    return int(lib().attn_cache_evict_workspace_size(batch, h_k, _int32("budget", budget),
                                                     _int32("max_seqlen", max_seqlen)))


def alloc_evict_workspace(seqlens, k_cache, budget: int, max_seqlen: int) -> torch.Tensor:
    """Workspace of attn_cache_evict for a batch of ``seqlens`` over ``k_cache``."""
    n = evict_workspace_size(seqlens.shape[0], k_cache.shape[2], budget, max_seqlen)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=seqlens.device)


def attn_cache_evict(k_cache, v_cache, block_table, seqlens, weights, budget: int, recent: int = 0,
                     slot_positions=None, seen=None, max_seqlen: Optional[int] = None,
                     weights_out=None, positions_out=None, seqlens_out=None, workspace=None,
                     stream=None):
    """Cuts every sequence to ``budget`` slots: returns (seqlens_out, weights_out, positions_out).

    Each head of a longer sequence keeps the slots whose token is among the
    ``recent`` newest (``slot_positions[b, h, j] >= seen[b] - recent``) and, for
    the rest, those of the largest ``weights`` (fp32 [B, H_k, >= max_seqlen], ties:
    the lower slot).  Kept slots at or above the budget move, in slot order, into
    the freed ones below; the order of the slots is then not that of the tokens,
    which attention over rotated keys does not depend on (a window does).  Caches
    are changed in place; ``weights_out`` and ``positions_out`` default to the
    inputs; slots [budget, seqlens[b]) get 0 and -1 there.  ``seqlens_out`` must
    not be ``seqlens``."""
    index, dtype, dt = _first(k_cache, "k_cache")
    batch = _batch(seqlens)
    cache, hk, d, slots = _cache(k_cache, v_cache, block_table, index, dtype, batch)
    lens = _ints("seqlens", seqlens, index, batch)
    max_seqlen = _int32("max_seqlen", slots if max_seqlen is None else max_seqlen)
    budget, recent = _int32("budget", budget), _int32("recent", recent)
    if weights_out is None:
        weights_out = weights
    w_in, width = _state("weights", weights, index, _F32, batch, hk, max_seqlen)
    w_out, same = _state("weights_out", weights_out, index, _F32, batch, hk, max_seqlen)
    p_in = p_out = None
    widths = {width, same}
    if slot_positions is not None:
        if positions_out is None:
            positions_out = slot_positions
        p_in, same = _state("slot_positions", slot_positions, index, _I32, batch, hk, max_seqlen)
        widths.add(same)
        p_out, same = _state("positions_out", positions_out, index, _I32, batch, hk, max_seqlen)
        widths.add(same)
    elif positions_out is not None:
        raise AttnError(-9, "positions_out without slot_positions")
    if len(widths) != 1:
        raise AttnError(-2, "weights, slot_positions and their outputs must have the same shape")
    side = _side(stream, index)
    if seqlens_out is None:
        seqlens_out = _new(side, torch.empty_like, seqlens)
    out = _ints("seqlens_out", seqlens_out, index, batch)
    if batch == 0:
        return seqlens_out, weights_out, positions_out
    ws, size, _held = _workspace(workspace, evict_workspace_size(batch, hk, budget, max_seqlen), k_cache,
                                 index, side)
    _call(lib().attn_cache_evict, index, stream, cache, dt, batch, hk, d, lens, out, max_seqlen,
          budget, recent, _ints("seen", seen, index, batch), w_in, w_out, p_in, p_out, width, ws, size)
    return seqlens_out, weights_out, positions_out
