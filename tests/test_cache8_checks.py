"""Refusals and the C boundary of the 8-bit cache and of shared pages (no GPU needed).

The C calls get made-up pointers, which only calls that are refused before any launch may get;
every case below differs from a valid call in one argument.
"""
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
from tests.test_cache_checks import T, rotary

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPE, SHAPE, STRIDE, ALIGN, NULL, WS, ARG = -1, -2, -3, -4, -5, -6, -9
P = 1 << 20
FACTORS = struct.Struct("@PPqqqqqqii")  # attn_paged_kv8 behind its attn_paged_kv


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return ab.lib()


def test_signatures_match_the_header(lib):
    text = open(os.path.join(ROOT, "include", "attn_cache8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    found = re.findall(r"([A-Za-z_][\w \t]*?\**)\s*\b(attn_[a-z0-9_]+)\s*\(([^()]*)\)\s*;", text)
    assert len(found) == 6
    for ret, name, params in found:
        f = getattr(lib, name)
        want = [_c_kind(p) for p in " ".join(params.split()).split(",")]
        assert [_ctypes_kind(t) for t in f.argtypes] == want, name
        assert _ctypes_kind(f.restype) == _c_kind(ret.strip() + " r"), name


def test_packed_structure_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ("kv", "k_scale", "v_scale", "k_scale_page", "k_scale_head", "v_scale_page", "v_scale_head", "block", "kind")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"attn_cache8.h\"\nint main(void) {\n"
                   "printf(\"size %zu\\n\", sizeof(attn_paged_kv8));\n" +
                   "\n".join(f'printf("{f} %zu\\n", offsetof(attn_paged_kv8, {f}));' for f in names) + "return 0;}\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    at = {x.split()[0]: int(x.split()[1]) for x in out.splitlines()}
    b = binding_cache._PAGED.pack(*range(1, 14)) + FACTORS.pack(*range(21, 31))
    assert len(b) == at["size"]
    assert at["kv"] == 0 and binding_cache._PAGED.size == at["k_scale"]
    for name, fmt, want in (("k_scale", "@P", 21), ("v_scale", "@P", 22), ("k_scale_page", "@q", 23),
                            ("k_scale_head", "@q", 25), ("v_scale_page", "@q", 26), ("v_scale_head", "@q", 28),
                            ("block", "@i", 29), ("kind", "@i", 30)):
        assert struct.unpack_from(fmt, b, at[name])[0] == want, name


def paged8(kptr=P, vptr=P, kh=64, ks=128, kb=2048, table=P, ts=8, pages=10, size=16, per=8, fk=P, fv=P, st=(4, 2, 1),
           vst=(4, 2, 1), block=8, kind=0):
    return binding_cache._PAGED.pack(kptr, kb, ks, kh, vptr, 2048, 128, 64, table, ts, pages, size, per) + \
        FACTORS.pack(fk, fv, *st, *vst, block, kind)


def append(lib, q=T(), oq=T(), k=T(), v=T(), dt=1, t=4, b=4, hq=2, hk=2, d=64, c=paged8(), n=P, cu=None, rot=rotary()):
    return lib.attn_cache_append8(q, oq, k, v, dt, t, b, hq, hk, d, c, n, cu, rot, None)


def load(lib, k=T(), v=T(), dt=1, t=4, b=4, hk=2, d=64, c=paged8(), at=P, cu=P):
    return lib.attn_cache_load8(k, v, dt, t, b, hk, d, c, at, cu, None)


def decode(lib, q=T(), o=T(), lse=P, dt=1, b=2, hq=4, hk=2, d=64, scale=0.1, c=paged8(), n=P, most=100, opts=None, ws=P,
           size=1 << 30):
    return lib.attn_decode8(q, o, lse, dt, b, hq, hk, d, scale, c, n, most, opts, ws, size, None)


A = [P + i * (1 << 16) for i in range(12)]


def fork(lib, tab=A[0], ts=8, tab2=A[1], ts2=8, n=A[2], n2=A[3], r=A[4], r2=A[5], pages=100, rows=4, per=8, page=16,
         who=A[6], room=A[7], all_=0, share=1, copies=A[8], counts=A[9], ws=A[10], size=1 << 16):
    return lib.attn_cache_fork(tab, ts, tab2, ts2, n, n2, r, r2, pages, rows, per, page, who, room, all_, share, copies,
                               counts, ws, size, None)


def copy(lib, c=paged8(), size=1, hk=2, d=64, pairs=P, count=None, n=3):
    return lib.attn_cache_copy(c, size, hk, d, pairs, count, n, None)


BAD_CACHE = [
    (dict(c=None), NULL), (dict(d=72), SHAPE), (dict(c=paged8(kind=2)), DTYPE), (dict(c=paged8(block=0)), SHAPE),
    (dict(c=paged8(block=3)), SHAPE), (dict(c=paged8(fk=0)), NULL), (dict(c=paged8(fv=0)), NULL),
    (dict(c=paged8(fk=P + 2)), ALIGN), (dict(c=paged8(st=(0, 2, 1))), STRIDE), (dict(c=paged8(vst=(4, -2, 1))), STRIDE),
    (dict(c=paged8(vst=(4, 2, 0))), STRIDE), (dict(c=paged8(st=(1 << 32, 2, 1))), STRIDE),
    (dict(c=paged8(vst=(4, 1 << 32, 1))), STRIDE), (dict(c=paged8(kh=72)), STRIDE), (dict(c=paged8(ks=136)), STRIDE),
    (dict(c=paged8(kb=-2048)), STRIDE), (dict(c=paged8(kptr=P + 8)), ALIGN), (dict(c=paged8(vptr=0)), NULL),
    (dict(c=paged8(table=0)), NULL), (dict(c=paged8(ts=7)), STRIDE), (dict(c=paged8(pages=0)), SHAPE),
    (dict(c=paged8(kb=1 << 40)), STRIDE), (dict(c=paged8(size=1 << 28, per=8)), SHAPE),
]
CASES = [(f, kw, code) for f in (append, load, decode) for kw, code in BAD_CACHE] + [
    (append, dict(dt=2), DTYPE), (append, dict(b=0, t=0), SHAPE), (append, dict(t=-1, cu=P), SHAPE),
    (append, dict(t=5), ARG), (append, dict(oq=None), ARG), (append, dict(rot=None), ARG),
    (append, dict(rot=rotary(inverse=1)), ARG), (append, dict(rot=rotary(n=33, sec=(33, 0, 0, 0))), SHAPE),
    (append, dict(n=None), NULL), (append, dict(n=P + 1), ALIGN), (append, dict(k=T(s=60)), STRIDE),
    (append, dict(v=T(ptr=0)), NULL), (append, dict(q=T(ptr=P + 4)), ALIGN),
    (append, dict(hk=1 << 29, hq=1 << 29), SHAPE),
    (load, dict(dt=3), DTYPE), (load, dict(t=-1), SHAPE), (load, dict(at=None), NULL), (load, dict(cu=None), NULL),
    (load, dict(cu=P + 2), ALIGN), (load, dict(k=T(ptr=0)), NULL), (load, dict(v=T(h=20)), STRIDE),
    (decode, dict(hq=3), SHAPE), (decode, dict(most=129), ARG), (decode, dict(most=-1), ARG),
    (decode, dict(n=None), NULL), (decode, dict(q=T(ptr=P + 8)), ALIGN), (decode, dict(o=T(ptr=0)), NULL),
    (decode, dict(lse=P + 2), ALIGN), (decode, dict(scale=float("nan")), ARG), (decode, dict(d=256 + 16), SHAPE),
    (decode, dict(opts=binding_cache._OPTS.pack(-2, -1, 0.0, 0, 0)), ARG),
    (decode, dict(opts=binding_cache._OPTS.pack(-1, -1, -1.0, 0, 0)), ARG),
    (decode, dict(opts=binding_cache._OPTS.pack(-1, -1, 0.0, 0, P)), ARG),
    (decode, dict(b=100, most=128, ws=None, hk=4, hq=8), WS), (decode, dict(b=100, hk=4, hq=8, ws=P + 128), WS),
    (decode, dict(b=100, hk=4, hq=8, size=256), WS),
    (fork, dict(rows=0), SHAPE), (fork, dict(pages=0), SHAPE), (fork, dict(page=0), SHAPE), (fork, dict(per=-1), SHAPE),
    (fork, dict(page=1 << 28), SHAPE), (fork, dict(rows=1 << 28, ts=1 << 20, ts2=1 << 20), SHAPE),
    (fork, dict(tab=None), NULL), (fork, dict(tab2=None), NULL), (fork, dict(n2=None), NULL), (fork, dict(r=None), NULL),
    (fork, dict(copies=None), NULL), (fork, dict(counts=None), NULL), (fork, dict(r2=A[5] + 2), ALIGN),
    (fork, dict(who=A[6] + 1), ALIGN), (fork, dict(ts=7), STRIDE), (fork, dict(ts2=7), STRIDE),
    (fork, dict(room=None, all_=-1), ARG), (fork, dict(tab2=A[0] + 4), ARG), (fork, dict(tab2=A[0], ts2=9), ARG),
    (fork, dict(r2=A[4] + 8), ARG), (fork, dict(n2=A[6]), ARG), (fork, dict(n2=A[7]), ARG), (fork, dict(copies=A[9]), ARG),
    (fork, dict(counts=A[4] + 16), ARG), (fork, dict(r2=A[1]), ARG), (fork, dict(ws=None), WS), (fork, dict(ws=A[10] + 4), WS),
    (fork, dict(size=64), WS),
    (copy, dict(c=None), NULL), (copy, dict(size=4), DTYPE), (copy, dict(d=72), SHAPE), (copy, dict(d=0), SHAPE),
    (copy, dict(hk=0), SHAPE), (copy, dict(c=paged8(size=1 << 28, block=1 << 28)), SHAPE), (copy, dict(n=-1), SHAPE), (copy, dict(pairs=None), NULL), (copy, dict(pairs=P + 2), ALIGN),
    (copy, dict(count=P + 1), ALIGN), (copy, dict(c=paged8(fk=0)), ARG), (copy, dict(c=paged8(block=5)), SHAPE),
    (copy, dict(c=paged8(kh=72)), STRIDE), (copy, dict(c=paged8(vptr=0)), NULL), (copy, dict(c=paged8(st=(4, 0, 1))), STRIDE),
]


@pytest.mark.parametrize("f,kw,code", CASES, ids=[f"{f.__name__}-{'-'.join(kw)}-{i}" for i, (f, kw, _) in enumerate(CASES)])
def test_bad_arguments_are_refused(lib, f, kw, code):
    assert f(lib, **kw) == code
    assert lib.attn_last_error()


def test_calls_without_work_launch_nothing(lib):
    assert append(lib, t=0, b=4, cu=P) == 0
    assert load(lib, t=0) == 0
    assert copy(lib, n=0, pairs=None) == 0


def test_workspace_sizes(lib):
    assert lib.attn_cache_fork_workspace_size(0, 8, 8) == 0
    assert lib.attn_cache_fork_workspace_size(1 << 20, 1 << 12, 8) == 0
    rows, per, pages = 5, 7, 20
    assert lib.attn_cache_fork_workspace_size(rows, per, pages) >= 4 * (7 * rows + pages + rows * per)


def test_binding_refuses_tensors_on_the_host():
    q, kc, table, n = torch.zeros(2, 4, 64).half(), torch.zeros(4, 8, 2, 64, dtype=torch.int8), \
        torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    s, k = torch.ones(4, 1, 2), torch.zeros(2, 2, 64).half()
    for call in (lambda: ab.attn_decode8(q, kc, kc, s, s, table, n), lambda: ab.attn_cache_append8(k, k, kc, kc, s, s, table, n),
                 lambda: ab.attn_cache_load8(kc, kc, s, s, table, n, torch.zeros(3, dtype=torch.int32), 4),
                 lambda: ab.attn_cache_fork(table, n, n, 8), lambda: ab.attn_cache_copy(kc, kc, table, k_scale=s, v_scale=s)):
        with pytest.raises(ab.AttnError):
            call()
