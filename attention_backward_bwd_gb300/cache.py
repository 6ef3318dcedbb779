"""Binding of the serving operators (include/attn_cache.h): rotary positions, the
paged key/value cache's append, attention of one new token over it, and eviction.

Argument marshalling only, like binding.py: every step of the computation runs in
the library's CUDA kernels, there is no fallback, and argument errors raise
AttnError before anything is launched.  Lengths, block tables and offsets live on
the device and are checked there; check_device_status() reports what was bad.

The calls run on the device of their tensors, on ``stream`` (default: that device's
current stream).
"""
from __future__ import annotations

import struct
from typing import Optional, Sequence, Tuple

import torch

from .binding import ATTN_BF16, ATTN_FP16, AttnError, lib

_DTYPES = {torch.float16: ATTN_FP16, torch.bfloat16: ATTN_BF16}
# attn_tensor, attn_paged_kv, attn_rotary and attn_opts as a C compiler lays them out
_TENSOR = struct.Struct("@Pqqq")
_PAGED = struct.Struct("@PqqqPqqqPqiii4x")
_ROTARY = struct.Struct("@PqPii4iii")
_OPTS = struct.Struct("@iif4xPP")


def _fail(rc: int):
    raise AttnError(rc, lib().attn_last_error().decode())


def _stream_of(stream, dev) -> int:
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(fn, dev, stream, made, *args):
    """Runs fn(*args, stream) with ``dev`` current.  ``made``: tensors allocated by
    the caller; their memory is kept from reuse until ``stream`` has passed them."""
    raw = _stream_of(stream, dev)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc != 0:
        _fail(rc)
    if stream is not None:
        other = stream if isinstance(stream, torch.cuda.Stream) else \
            torch.cuda.ExternalStream(raw, device=dev)
        for t in made:
            t.record_stream(other)


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise AttnError(-1, f"{name} must be float16 or bfloat16, got {t.dtype}")
    return code


def _rows(name, t, like, dims) -> None:
    """Device, dtype, rank and a unit stride over the head dimension."""
    if not t.is_cuda or t.device != like.device:
        raise AttnError(-9, f"{name} must be a CUDA tensor on {like.device}, got {t.device}")
    if t.dtype != like.dtype:
        raise AttnError(-1, f"{name} has dtype {t.dtype}, {like.dtype} was expected")
    if t.dim() != dims:
        raise AttnError(-2, f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.numel() > 0:
        raise AttnError(-3, f"{name} must have unit stride over the head dimension")


def _ints(name, t, dev, shape) -> int:
    """Pointer of a contiguous int32 tensor of the given shape (or None)."""
    if t is None:
        return 0
    if t.device != dev or t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise AttnError(-9, f"{name} must be a contiguous int32 tensor of shape {shape} on {dev}, "
                            f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _state(name, t, dev, dtype, batch, heads, width) -> int:
    """Pointer of a contiguous [batch, H_k, >= width] tensor of per-slot state."""
    s = t.shape
    if t.device != dev or t.dtype != dtype or len(s) != 3 or s[0] != batch or s[1] != heads or \
            s[2] < width or not t.is_contiguous():
        raise AttnError(-9, f"{name} must be a contiguous {dtype} tensor [{batch}, {heads}, >= {width}] "
                            f"on {dev}, got {t.dtype} {tuple(s)} on {t.device}")
    return t.data_ptr()


def _cache(k_cache, v_cache, table, like, batch) -> Tuple[bytes, int, int]:
    """(attn_paged_kv, H_k, slots of a sequence)."""
    _rows("k_cache", k_cache, like, 4)
    _rows("v_cache", v_cache, like, 4)
    pages, size, heads, _ = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise AttnError(-2, f"v_cache has shape {tuple(v_cache.shape)}, k_cache {tuple(k_cache.shape)}")
    if table.device != like.device or table.dtype != torch.int32 or table.dim() != 2 or \
            table.shape[0] != batch or (table.shape[1] > 1 and table.stride(1) != 1):
        raise AttnError(-9, f"block_table must be an int32 tensor [{batch}, pages] on {like.device} with "
                            f"contiguous rows, got {table.dtype} {tuple(table.shape)} on {table.device}")
    ks, vs = k_cache.stride(), v_cache.stride()
    per = table.shape[1]
    return _PAGED.pack(k_cache.data_ptr(), ks[0], ks[1], ks[2], v_cache.data_ptr(), vs[0], vs[1], vs[2],
                       table.data_ptr(), table.stride(0), pages, size, per), heads, per * size


def _rotary(positions, inv_freq, sections, interleaved, inverse, dev, lead) -> bytes:
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.device != dev or \
            inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise AttnError(-9, f"inv_freq must be a contiguous 1-D float32 tensor on {dev}")
    n = inv_freq.shape[0]
    sec = (n,) if sections is None else tuple(int(x) for x in sections)
    if not 1 <= len(sec) <= 4:
        raise AttnError(-2, f"sections must name 1 to 4 axes, got {len(sec)}")
    shape = tuple(positions.shape)
    if shape != (len(sec),) + lead and not (len(sec) == 1 and shape == lead):
        raise AttnError(-2, f"positions must be {(len(sec),) + lead}, got {shape}")
    if positions.device != dev or positions.dtype != torch.int32 or not positions.is_contiguous():
        raise AttnError(-9, f"positions must be a contiguous int32 tensor on {dev}, got "
                            f"{positions.dtype} on {positions.device}")
    tokens = 1
    for x in lead:
        tokens *= x
    return _ROTARY.pack(positions.data_ptr(), tokens, inv_freq.data_ptr(), n, len(sec),
                        *(sec + (0, 0, 0, 0))[:4], int(bool(interleaved)), int(bool(inverse)))


def _pack(t, packed: bool) -> bytes:
    s = t.stride()
    return _TENSOR.pack(t.data_ptr(), 0, s[0], s[1]) if packed else \
        _TENSOR.pack(t.data_ptr(), s[0], s[1], s[2])


def _same_place(name, out, x) -> None:
    if out.data_ptr() == x.data_ptr() and out.numel() > 0 and out.stride() != x.stride():
        raise AttnError(-9, f"{name} starts where its input does but has other strides")


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
    L = lib()
    if q.dim() not in (3, 4):
        raise AttnError(-2, f"q must be [B, S, H, D] or packed [total, H, D], got {tuple(q.shape)}")
    packed = q.dim() == 3
    dt = _dtype(q, "q")
    _rows("q", q, q, q.dim())
    dev, lead = q.device, tuple(q.shape[:-2])
    made = []
    if out_q is None:
        out_q = torch.empty_like(q)
        made.append(out_q)
    if k is not None:
        _rows("k", k, q, q.dim())
        if tuple(k.shape[:-2]) != lead or k.shape[-1] != q.shape[-1]:
            raise AttnError(-2, f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree on tokens or D")
        if out_k is None:
            out_k = torch.empty_like(k)
            made.append(out_k)
    elif out_k is not None:
        raise AttnError(-9, "out_k without k")
    for name, out, x in (("out_q", out_q, q), ("out_k", out_k, k)):
        if x is not None and not (made and out is made[0]):
            _rows(name, out, q, q.dim())
            if out.shape != x.shape:
                raise AttnError(-2, f"{name} has shape {tuple(out.shape)}, its input {tuple(x.shape)}")
            _same_place(name, out, x)
    rot = _rotary(positions, inv_freq, sections, interleaved, inverse, dev, lead)
    batch, seqlen = (1, lead[0]) if packed else lead
    if batch == 0 or seqlen == 0:
        return out_q, out_k
    _call(L.attn_rope, dev, stream, made, _pack(q, packed), None if k is None else _pack(k, packed),
          _pack(out_q, packed), None if k is None else _pack(out_k, packed), dt, batch, seqlen,
          q.shape[-2], q.shape[-2] if k is None else k.shape[-2], q.shape[-1], rot)
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
    L = lib()
    dt = _dtype(k, "k")
    _rows("k", k, k, 3)
    _rows("v", v, k, 3)
    dev = k.device
    tokens, hk, d = k.shape
    if v.shape != k.shape:
        raise AttnError(-2, f"v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
    batch = seqlens.shape[0] if seqlens.dim() == 1 else -1
    lens = _ints("seqlens", seqlens, dev, (batch,))
    cache, heads, slots = _cache(k_cache, v_cache, block_table, k, batch)
    if heads != hk or k_cache.shape[3] != d:
        raise AttnError(-2, f"k {tuple(k.shape)} does not fit a cache {tuple(k_cache.shape)}")
    cu = _ints("cu_seqlens", cu_seqlens, dev, (batch + 1,))
    if cu_seqlens is None and tokens != batch:
        raise AttnError(-9, f"without cu_seqlens there is one token a sequence: {tokens} tokens, "
                            f"{batch} sequences")
    if (positions is None) != (inv_freq is None):
        raise AttnError(-9, "positions and inv_freq go together")
    rot = None if positions is None else \
        _rotary(positions, inv_freq, sections, interleaved, False, dev, (tokens,))
    made = []
    q_arg = oq_arg = None
    hq = hk
    if q is not None:
        if rot is None:
            raise AttnError(-9, "q is only taken to be rotated: give positions and inv_freq, or no q")
        _rows("q", q, k, 3)
        if q.shape[0] != tokens or q.shape[2] != d:
            raise AttnError(-2, f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree on tokens or D")
        if out_q is None:
            out_q = torch.empty_like(q)
            made.append(out_q)
        else:
            _rows("out_q", out_q, k, 3)
            if out_q.shape != q.shape:
                raise AttnError(-2, f"out_q has shape {tuple(out_q.shape)}, q {tuple(q.shape)}")
            _same_place("out_q", out_q, q)
        hq = q.shape[1]
        q_arg, oq_arg = _pack(q, True), _pack(out_q, True)
    elif out_q is not None:
        raise AttnError(-9, "out_q without q")
    sp, width = 0, 0
    if slot_positions is not None:
        if seen is None:
            raise AttnError(-9, "slot_positions needs seen")
        sp = _state("slot_positions", slot_positions, dev, torch.int32, batch, hk, 1)
        width = slot_positions.shape[2]
    if tokens == 0:
        return out_q
    _call(L.attn_cache_append, dev, stream, made, q_arg, oq_arg, _pack(k, True), _pack(v, True), dt,
          tokens, batch, hq, hk, d, cache, lens, cu or None, rot, sp or None, width,
          _ints("seen", seen, dev, (batch,)) or None)
    return out_q


def decode_workspace_size(batch: int, h_q: int, h_k: int, head_dim: int, max_seqlen: int,
                          weights: bool = False) -> int:
    return int(lib().attn_decode_workspace_size(batch, h_q, h_k, head_dim, max_seqlen, int(weights)))


def alloc_decode_workspace(q, k_cache, max_seqlen: int, weights: bool = False) -> torch.Tensor:
    """Workspace of attn_decode for queries like ``q`` [B, H_q, D] over ``k_cache``."""
    n = decode_workspace_size(q.shape[0], q.shape[1], k_cache.shape[2], q.shape[2], max_seqlen, weights)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def _workspace(workspace, need, dev, made) -> torch.Tensor:
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise AttnError(-9, f"workspace must be a contiguous uint8 tensor on {dev}")
    return workspace


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
    L = lib()
    dt = _dtype(q, "q")
    _rows("q", q, q, 3)
    dev = q.device
    batch, hq, d = q.shape
    cache, hk, slots = _cache(k_cache, v_cache, block_table, q, batch)
    if k_cache.shape[3] != d or hq % max(hk, 1) != 0:
        raise AttnError(-2, f"q {tuple(q.shape)} does not fit a cache {tuple(k_cache.shape)}")
    lens = _ints("seqlens", seqlens, dev, (batch,))
    max_seqlen = slots if max_seqlen is None else int(max_seqlen)
    made = []
    if out is None:
        out = torch.empty_like(q)
        made.append(out)
    else:
        _rows("out", out, q, 3)
        if out.shape != q.shape:
            raise AttnError(-2, f"out has shape {tuple(out.shape)}, q {tuple(q.shape)}")
    if lse is None:
        lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)
        made.append(lse)
    elif lse.device != dev or lse.dtype != torch.float32 or tuple(lse.shape) != (batch, hq) or \
            not lse.is_contiguous():
        raise AttnError(-2, f"lse must be a contiguous float32 tensor {(batch, hq)} on {dev}")
    if batch == 0:
        return out, lse
    w_in = w_out = None
    width = 0
    if weights is not None:
        weights_out = weights if weights_out is None else weights_out
        w_in = _state("weights", weights, dev, torch.float32, batch, hk, max_seqlen)
        w_out = _state("weights_out", weights_out, dev, torch.float32, batch, hk, max_seqlen)
        width = weights.shape[2]
        if weights_out.shape[2] != width:
            raise AttnError(-2, "weights and weights_out must have the same shape")
    elif weights_out is not None:
        raise AttnError(-9, "weights_out without weights")
    need = L.attn_decode_workspace_size(batch, hq, hk, d, max_seqlen, weights is not None)
    workspace = _workspace(workspace, need, dev, made)
    opts = None
    if window is not None or softcap:
        left, right = (-1, -1) if window is None else (int(window[0]), int(window[1]))
        opts = _OPTS.pack(left, right, float(softcap or 0.0), 0, 0)
    qs, os = q.stride(), out.stride()
    _call(L.attn_decode, dev, stream, made, _TENSOR.pack(q.data_ptr(), qs[0], 0, qs[1]),
          _TENSOR.pack(out.data_ptr(), os[0], 0, os[1]), lse.data_ptr(), dt, batch, hq, hk, d,
          d ** -0.5 if scale is None else float(scale), cache, lens, max_seqlen, opts, w_in, w_out,
          width, workspace.data_ptr(), workspace.numel())
    return out, lse


def evict_workspace_size(batch: int, h_k: int, budget: int, max_seqlen: int) -> int:
    return int(lib().attn_cache_evict_workspace_size(batch, h_k, budget, max_seqlen))


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
    L = lib()
    dt = _dtype(k_cache, "k_cache")
    dev = k_cache.device
    batch = seqlens.shape[0] if seqlens.dim() == 1 else -1
    cache, hk, slots = _cache(k_cache, v_cache, block_table, k_cache, batch)
    lens = _ints("seqlens", seqlens, dev, (batch,))
    max_seqlen = slots if max_seqlen is None else int(max_seqlen)
    weights_out = weights if weights_out is None else weights_out
    w_in = _state("weights", weights, dev, torch.float32, batch, hk, max_seqlen)
    w_out = _state("weights_out", weights_out, dev, torch.float32, batch, hk, max_seqlen)
    width = weights.shape[2]
    p_in = p_out = None
    same = weights_out.shape[2] == width
    if slot_positions is not None:
        positions_out = slot_positions if positions_out is None else positions_out
        p_in = _state("slot_positions", slot_positions, dev, torch.int32, batch, hk, max_seqlen)
        p_out = _state("positions_out", positions_out, dev, torch.int32, batch, hk, max_seqlen)
        same = same and slot_positions.shape[2] == width and positions_out.shape[2] == width
    elif positions_out is not None:
        raise AttnError(-9, "positions_out without slot_positions")
    if not same:
        raise AttnError(-2, "weights, slot_positions and their outputs must have the same shape")
    made = []
    if seqlens_out is None:
        seqlens_out = torch.empty_like(seqlens)
        made.append(seqlens_out)
    out = _ints("seqlens_out", seqlens_out, dev, (batch,))
    if batch == 0:
        return seqlens_out, weights_out, positions_out
    need = L.attn_cache_evict_workspace_size(batch, hk, int(budget), max_seqlen)
    workspace = _workspace(workspace, need, dev, made)
    _call(L.attn_cache_evict, dev, stream, made, cache, dt, batch, hk, k_cache.shape[3], lens, out,
          max_seqlen, int(budget), int(recent), _ints("seen", seen, dev, (batch,)) or None, w_in, w_out,
          p_in, p_out, width, workspace.data_ptr(), workspace.numel())
    return seqlens_out, weights_out, positions_out
