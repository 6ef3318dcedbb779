"""Refusals and the C boundary of the serving operators (no GPU needed).

The C calls get made-up pointers, which only calls that are refused before any
launch may get; every case below differs from a valid call in one argument.
"""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import attention_backward_bwd_gb300 as ab
from attention_backward_bwd_gb300 import cache as binding_cache
from tests.test_abi_host import _c_kind, _ctypes_kind

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPE, SHAPE, STRIDE, ALIGN, NULL, WS, ARG = -1, -2, -3, -4, -5, -6, -9
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return ab.lib()


def header():
    text = open(os.path.join(ROOT, "include", "attn_cache.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_signatures_match_the_header(lib):
    found = re.findall(r"([A-Za-z_][\w \t]*?\**)\s*\b(attn_[a-z0-9_]+)\s*\(([^()]*)\)\s*;", header())
    assert len(found) == 6
    for ret, name, params in found:
        f = getattr(lib, name)
        want = [_c_kind(p) for p in " ".join(params.split()).split(",")]
        assert [_ctypes_kind(t) for t in f.argtypes] == want, name
        assert _ctypes_kind(f.restype) == _c_kind(ret.strip() + " r"), name


def test_packed_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = {"attn_tensor": ("ptr", "stride_b", "stride_s", "stride_h"),
              "attn_paged_kv": ("k", "v", "block_table", "table_stride", "num_pages", "page_size", "max_pages"),
              "attn_rotary": ("positions", "axis_stride", "inv_freq", "n_freq", "n_axes", "sections",
                              "interleaved", "inverse"),
              "attn_opts": ("window_left", "window_right", "softcap", "seqused_q", "seqused_k")}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "attn_cache.h"', "int main(void) {"]
    for st, fs in fields.items():
        lines.append(f'  printf("{st} size %zu\\n", sizeof({st}));')
        lines += [f'  printf("{st} {f} %zu\\n", offsetof({st}, {f}));' for f in fs]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    c = {tuple(x.split()[:2]): int(x.split()[2]) for x in out.splitlines()}
    packs = {"attn_tensor": (binding_cache._TENSOR, "PPPP"), "attn_opts": (binding_cache._OPTS, None),
             "attn_paged_kv": (binding_cache._PAGED, None), "attn_rotary": (binding_cache._ROTARY, None)}
    for st, (pk, _) in packs.items():
        assert pk.size == c[(st, "size")], st
    b = binding_cache._PAGED.pack(*range(1, 14))
    at = lambda st, f, fmt: struct.unpack_from(fmt, b, c[(st, f)])[0]  # noqa: E731
    assert at("attn_paged_kv", "v", "@P") == 5 and at("attn_paged_kv", "block_table", "@P") == 9
    assert at("attn_paged_kv", "num_pages", "@i") == 11 and at("attn_paged_kv", "max_pages", "@i") == 13
    b = binding_cache._ROTARY.pack(*range(1, 12))
    assert at("attn_rotary", "inv_freq", "@P") == 3 and at("attn_rotary", "n_axes", "@i") == 5
    assert at("attn_rotary", "sections", "@i") == 6 and at("attn_rotary", "inverse", "@i") == 11


def T(ptr=P, b=64 * 64, s=64, h=64):
    return binding_cache._TENSOR.pack(ptr, b, s, h)


def paged(kptr=P, vptr=P, kh=64, table=P, ts=8, pages=10, size=16, per=8):
    return binding_cache._PAGED.pack(kptr, 2048, 128, kh, vptr, 2048, 128, 64, table, ts, pages, size, per)


def rotary(pos=P, axis=100, inv=P, n=32, axes=1, sec=(32, 0, 0, 0), inverse=0):
    return binding_cache._ROTARY.pack(pos, axis, inv, n, axes, *sec, 0, inverse)


def rope(lib, q=T(), k=T(), oq=T(), ok=T(), dt=1, b=2, s=40, hq=2, hk=2, d=64, rot=rotary()):
    return lib.attn_rope(q, k, oq, ok, dt, b, s, hq, hk, d, rot, None)


def append(lib, q=T(), oq=T(), k=T(), v=T(), dt=1, t=4, b=4, hq=2, hk=2, d=64, c=paged(), n=P, cu=None,
           rot=rotary(), sp=None, width=0, seen=None):
    return lib.attn_cache_append(q, oq, k, v, dt, t, b, hq, hk, d, c, n, cu, rot, sp, width, seen, None)


def decode(lib, q=T(), o=T(), lse=P, dt=1, b=2, hq=4, hk=2, d=64, scale=0.1, c=paged(), n=P, most=100, opts=None,
           wi=None, wo=None, width=0, ws=P, size=1 << 30):
    return lib.attn_decode(q, o, lse, dt, b, hq, hk, d, scale, c, n, most, opts, wi, wo, width, ws, size, None)


def evict(lib, c=paged(), dt=1, b=2, hk=2, d=64, n=P, n2=2 * P, most=100, budget=50, recent=0, seen=None, wi=P, wo=P,
          pi=None, po=None, width=100, ws=P, size=1 << 30):
    return lib.attn_cache_evict(c, dt, b, hk, d, n, n2, most, budget, recent, seen, wi, wo, pi, po, width, ws,
                                size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), DTYPE), (dict(d=60), SHAPE), (dict(d=264), SHAPE), (dict(hq=3), SHAPE), (dict(s=-1), SHAPE),
    (dict(b=0), SHAPE), (dict(b=1 << 16, s=1 << 16), SHAPE),
    (dict(q=T(0)), NULL), (dict(oq=T(0)), NULL), (dict(ok=T(0)), NULL), (dict(q=T(P + 8)), ALIGN),
    (dict(ok=T(P + 2)), ALIGN), (dict(oq=T(h=0)), STRIDE), (dict(k=T(s=-64)), STRIDE), (dict(q=T(b=4)), STRIDE),
    (dict(rot=None), NULL), (dict(rot=rotary(n=33, sec=(33, 0, 0, 0))), SHAPE), (dict(rot=rotary(n=0, sec=(0,) * 4)), SHAPE),
    (dict(rot=rotary(axes=0)), SHAPE), (dict(rot=rotary(axes=5)), SHAPE), (dict(rot=rotary(sec=(31, 0, 0, 0))), SHAPE),
    (dict(rot=rotary(axes=2, sec=(40, -8, 0, 0))), SHAPE), (dict(rot=rotary(pos=0)), NULL),
    (dict(rot=rotary(inv=0)), NULL), (dict(rot=rotary(inv=P + 1)), ALIGN),
    (dict(rot=rotary(axes=2, sec=(16, 16, 0, 0), axis=79)), STRIDE),
])
def test_rope_refuses(lib, kw, code):
    assert rope(lib, **kw) == code, lib.attn_last_error()
    assert lib.attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), DTYPE), (dict(t=-1), SHAPE), (dict(t=5), ARG), (dict(q=None), ARG), (dict(oq=None), ARG),
    (dict(rot=None), ARG), (dict(rot=rotary(inverse=1)), ARG), (dict(n=None), NULL), (dict(n=P + 2), ALIGN),
    (dict(c=None), NULL), (dict(c=paged(kptr=0)), NULL), (dict(c=paged(vptr=P + 8)), ALIGN),
    (dict(c=paged(kh=4)), STRIDE), (dict(c=paged(table=0)), NULL), (dict(c=paged(ts=7)), STRIDE),
    (dict(c=paged(pages=0)), SHAPE), (dict(c=paged(size=0)), SHAPE), (dict(c=paged(size=1 << 29)), SHAPE),
    (dict(sp=P, width=9), NULL), (dict(sp=P, width=0, seen=P), STRIDE), (dict(sp=P + 1, width=9, seen=P), ALIGN),
    (dict(k=T(0)), NULL), (dict(v=T(P + 4)), ALIGN), (dict(hq=3), SHAPE),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code, lib.attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), DTYPE), (dict(hq=5), SHAPE), (dict(d=4), SHAPE), (dict(scale=float("nan")), ARG),
    (dict(most=-1), ARG), (dict(most=129), ARG), (dict(q=T(0)), NULL), (dict(o=T(P + 8)), ALIGN),
    (dict(o=T(h=0)), STRIDE), (dict(n=None), NULL), (dict(lse=P + 2), ALIGN), (dict(wi=P, width=100), ARG),
    (dict(wi=P, wo=P, width=99), STRIDE),
    # (up to 256 keys need no workspace)
    (dict(ws=None, most=300, c=paged(per=20, ts=20)), WS), (dict(ws=P + 64, most=300, c=paged(per=20, ts=20)), WS),
    (dict(size=3, most=300, c=paged(per=20, ts=20)), WS), (dict(ws=None, wi=P, wo=P, width=100), WS),
    (dict(opts=binding_cache._OPTS.pack(-2, -1, 0.0, 0, 0)), ARG),
    (dict(opts=binding_cache._OPTS.pack(-1, -1, -1.0, 0, 0)), ARG),
    (dict(opts=binding_cache._OPTS.pack(-1, -1, 0.0, 0, P)), ARG),
])
def test_decode_refuses(lib, kw, code):
    assert decode(lib, **kw) == code, lib.attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), DTYPE), (dict(budget=0), ARG), (dict(recent=-1), ARG), (dict(recent=51), ARG),
    (dict(most=129, width=200), ARG), (dict(n=None), NULL), (dict(n2=None), NULL), (dict(n2=P), ARG),
    (dict(wi=None), NULL), (dict(wo=None), NULL), (dict(pi=P), ARG), (dict(recent=1), ARG),
    (dict(recent=1, pi=P, po=P), ARG), (dict(width=99), STRIDE), (dict(wo=P + 2), ALIGN), (dict(ws=None), WS),
    (dict(size=16), WS), (dict(b=0), SHAPE),
])
def test_evict_refuses(lib, kw, code):
    assert evict(lib, **kw) == code, lib.attn_last_error()


def test_workspace_sizes(lib):
    a = ab.decode_workspace_size(4, 32, 8, 128, 1000)
    b = ab.decode_workspace_size(4, 32, 8, 128, 1000, weights=True)
    assert a > 0 and a % 256 == 0 and b >= a + 4 * 32 * 1000 * 4
    assert ab.decode_workspace_size(4, 5, 2, 128, 10) == 0
    assert ab.decode_workspace_size(4, 32, 8, 128, 256) == 0
    assert ab.decode_workspace_size(4, 32, 8, 128, 100, weights=True) > 0
    # a head's sources and targets: at most as many as the budget, and as the slots above it
    assert ab.evict_workspace_size(4, 8, 100, 1000) == 4 * 8 * 2 * 100 * 4
    assert ab.evict_workspace_size(4, 8, 900, 1000) == 4 * 8 * 2 * 100 * 4
    assert ab.evict_workspace_size(4, 8, 100, 50) >= 4 * 8 * 4
    assert ab.evict_workspace_size(0, 8, 100, 50) == 0


def _code(fn, *a, **kw):
    with pytest.raises(ab.AttnError) as e:
        fn(*a, **kw)
    return e.value.code


def test_python_entry_points_refuse_what_is_not_on_a_gpu(lib):
    q = torch.randn(4, 2, 64).half()
    c = torch.randn(6, 16, 2, 64).half()
    table, n = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    pos, inv = torch.zeros(4, dtype=torch.int32), torch.ones(32)
    assert _code(ab.attn_rope, q, q, pos, inv) == ARG
    assert _code(ab.attn_cache_append, q, q, c, c, table, n) == ARG
    assert _code(ab.attn_decode, q, c, c, table, n) == ARG
    assert _code(ab.attn_cache_evict, c, c, table, n, torch.zeros(4, 2, 16), 4) == ARG
    assert _code(ab.attn_rope, q.float(), None, pos, inv) == DTYPE
    assert _code(ab.attn_decode, q.to("meta"), c, c, table, n) == ARG


def test_evict_refuses_lengths_that_overlap(lib):
    for n2 in (P, P + 4, P - 4):
        assert evict(lib, n2=n2) == ARG, n2           # b = 2: seqlens is [P, P + 8)
    for n2 in (2 * P, 2 * P + 4, 2 * P - 4):
        assert evict(lib, n2=n2, recent=1, seen=2 * P, pi=P, po=P) == ARG, n2
    assert evict(lib, n2=P + 8, ws=None) == WS        # beside it: refused for the next reason


def test_integers_beyond_32_bits_are_refused(lib):
    for bad in (2**31, 2**32 + 5, -2**31 - 1):
        assert _code(binding_cache._int32, "x", bad) == ARG
        assert _code(binding_cache._pack, binding_cache._OPTS, bad, 0, 0.0, 0, 0) == ARG
        assert _code(ab.decode_workspace_size, 4, 32, 8, 128, bad) == ARG
        assert _code(ab.evict_workspace_size, 4, 8, bad, 100) == ARG
    assert binding_cache._int32("x", 2**31 - 1) == 2**31 - 1


def test_lengths_next_to_2_to_the_31_are_refused(lib):
    """Tiles and runs of slots are counted in 32 bits: from 2^31 - 8191 on they could pass them."""
    last, wide = 2**31 - 8192, paged(size=1, per=2**31 - 1, ts=2**31 - 1)
    for most in (last + 1, 2**31 - 64, 2**31 - 1):
        assert decode(lib, c=wide, most=most, ws=None) == ARG, most
        assert decode(lib, c=wide, most=most, wi=P, wo=P, width=2**31, ws=None) == ARG, most
        assert evict(lib, c=wide, most=most, width=2**31, ws=None) == ARG, most
        assert lib.attn_decode_workspace_size(1, 1, 1, 64, most, 1) == 0
        assert lib.attn_cache_evict_workspace_size(1, 1, 100, most) == 0
    # the longest one allowed is refused for the next reason, and its workspace holds its logits
    assert decode(lib, c=wide, most=last, ws=None) == WS
    assert evict(lib, c=wide, most=last, width=2**31, ws=None) == WS
    assert lib.attn_decode_workspace_size(1, 1, 1, 64, last, 1) >= 4 * last
    assert lib.attn_cache_evict_workspace_size(1, 1, 2**30, last) >= 8 * (last - 2**30)
