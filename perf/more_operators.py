"""Cases and plain forms of the operators of a cache held in 8 bits and of shared pages: the append that
quantises, the read-back, single-token attention over 8-bit pages, forking and freeing of sequences, and
the copy of pages.

``run`` takes what ``prepare`` made and makes one pass through one operator (an append reads back what
it changed, which is how its values are seen): in plain torch operations where ``own`` is false, through
the package's entry points where it is true.  ``exact`` computes the same outputs in 64 bits, apart from
the plain form.

The cache: codes of 8 bits [pages, page, heads, dim], e4m3 or int8, and a factor in 32 bits for each block
of tokens of a page and head, [pages, page / block, heads], a power of two in 2^-60 .. 2^60.  An append
takes the smallest such factor with which no new value of the block is above 448 (int8: 127) of it, but not
less than the factor of the block's earlier tokens; where it grows they are rounded to it again.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
KIND = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
DEV = "cuda"
INF = float("inf")


def listed():
    return [
        # a decode step of a batch of chats: one token each enters blocks that hold some, q rotated in the same call
        {"name": "append8_step", "op": "append", "dtype": "bf16", "kind": "e4m3", "batch": 64, "lo": 100, "hi": 2000,
         "new_lo": 1, "new_hi": 1, "hq": 32, "hk": 8, "dim": 128, "rotary": 128, "axes": 1, "interleaved": False,
         "page": 64, "block": 16, "heads_first": False},
        # ragged prompts entering the cache, blocks of a whole page, part of the head rotated
        {"name": "append8_prompts", "op": "append", "dtype": "fp16", "kind": "int8", "batch": 16, "lo": 0, "hi": 300,
         "new_lo": 128, "new_hi": 2048, "hq": 16, "hk": 16, "dim": 96, "rotary": 64, "axes": 2, "interleaved": True,
         "page": 32, "block": 32, "heads_first": True},
        # prefixes that the next chunk of each prompt attends with the forward kernel
        {"name": "load8_prefix", "op": "load", "dtype": "bf16", "kind": "e4m3", "batch": 8, "lo": 0, "hi": 0,
         "new_lo": 1000, "new_hi": 8192, "hk": 8, "dim": 128, "page": 64, "block": 16, "heads_first": False},
        # the newest tokens of a few short sequences
        {"name": "load8_short", "op": "load", "dtype": "fp16", "kind": "int8", "batch": 5, "lo": 3, "hi": 90,
         "new_lo": 1, "new_hi": 77, "hk": 4, "dim": 80, "page": 24, "block": 8, "heads_first": True},
        # one short chat on small heads: latency alone
        {"name": "decode8_smallest", "op": "decode", "dtype": "fp16", "kind": "e4m3", "batch": 1, "lo": 128, "hi": 128,
         "hq": 2, "hk": 2, "dim": 64, "page": 16, "block": 16, "window": -1, "cap": 0.0, "heads_first": False},
        # one user with a very long document: the length has to be split
        {"name": "decode8_long", "op": "decode", "dtype": "bf16", "kind": "int8", "batch": 1, "lo": 131071, "hi": 131071,
         "hq": 32, "hk": 8, "dim": 128, "page": 128, "block": 128, "window": -1, "cap": 0.0, "heads_first": True},
        # the largest batch of long chats
        {"name": "decode8_largest", "op": "decode", "dtype": "bf16", "kind": "e4m3", "batch": 64, "lo": 4096, "hi": 16384,
         "hq": 32, "hk": 8, "dim": 128, "page": 64, "block": 16, "window": -1, "cap": 0.0, "heads_first": False},
        # wide heads without sharing, a sliding window and a logit cap, pages of an odd size
        {"name": "decode8_window_cap", "op": "decode", "dtype": "fp16", "kind": "int8", "batch": 9, "lo": 1, "hi": 4096,
         "hq": 16, "hk": 16, "dim": 256, "page": 48, "block": 24, "window": 1024, "cap": 30.0, "heads_first": False},
        # a step of a beam search: beams of 4 change places, each makes room for its next token
        {"name": "fork_beams", "op": "fork", "batch": 64, "beams": 4, "lo": 60, "hi": 4000, "page": 64, "spare": 512,
         "room": 1, "ended": False, "share": True},
        # a large pool: some sequences have ended, others start many samples on long prompts
        {"name": "fork_pool", "op": "fork", "batch": 512, "beams": 16, "lo": 1000, "hi": 16384, "page": 16, "spare": 60000,
         "room": 16, "ended": True, "share": True},
        # the last pages of the beams, in 16 bits, each page's heads one after the other
        {"name": "copy_beams", "op": "copy", "dtype": "bf16", "kind": "", "pages": 1024, "pairs": 48, "page": 64, "hk": 8,
         "dim": 128, "block": 64, "heads_first": True},
        # whole sequences copied in 8 bits with their factors
        {"name": "copy8_sequences", "op": "copy", "dtype": "", "kind": "e4m3", "pages": 12000, "pairs": 4000, "page": 64,
         "hk": 8, "dim": 128, "block": 16, "heads_first": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _divisor(rng, n):
    return rng.choice([d for d in range(1, n + 1) if n % d == 0])


def draw(rng):
    op = rng.choice(["append", "load", "decode", "decode", "fork", "copy"])
    if op == "fork":
        c = {"op": op, "batch": _log(rng, 1, 512), "beams": rng.choice([1, 2, 3, 4, 8, 16]),
             "page": rng.choice([1, 8, 16, 16, 32, 48, 64, 100, 128, 256]), "room": rng.choice([0, 1, 1, 16, 100]),
             "ended": rng.random() < 0.5, "share": rng.random() < 0.8, "spare": _log(rng, 1, 60000)}
        hi = max(1, min(_log(rng, 1, 16384), 1000 * c["page"], 400000 * c["page"] // c["batch"]))
        c.update(lo=rng.choice([0, 1, hi // 2]), hi=hi)
        return c
    hk = rng.choice([1, 2, 4, 8, 16])
    page = rng.choice([1, 8, 16, 16, 32, 48, 64, 100, 128, 256])
    c = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "kind": rng.choice(["e4m3", "int8"]), "hk": hk,
         "dim": rng.choice([16, 64, 64, 80, 96, 112, 128, 128, 144, 192, 256]), "page": page,
         "block": rng.choice([page, _divisor(rng, page)]), "heads_first": rng.random() < 0.5}
    if op == "copy":
        if rng.random() < 0.4:
            c.update(kind="", block=page)
        else:
            c.update(dtype="")
        c["pages"] = max(2, min(_log(rng, 2, 12000), 786432000 // (page * hk * c["dim"])))
        c["pairs"] = max(1, min(_log(rng, 1, 4000), c["pages"] // 2, 262144000 // (page * hk * c["dim"])))
        return c
    group = rng.choice([1, 2, 3, 4, 5, 8, 16, 20]) if hk <= 8 else rng.choice([1, 2])
    if op == "decode":
        batch, hi = _log(rng, 1, 128), _log(rng, 1, 131072)
        hi = max(1, min(hi, 80000000 // (batch * hk * c["dim"] // 8)))
        c.update(batch=batch, lo=rng.choice([0, 1, max(1, hi // 2)]) if batch > 1 else max(1, hi // 2), hi=hi,
                 hq=hk * group, window=rng.choice([-1, -1, _log(rng, 1, 4096)]), cap=rng.choice([0.0, 0.0, 20.0]))
        return c
    hi = rng.choice([1, 1, _log(rng, 1, 2048)]) if op == "append" else _log(rng, 1, 8192)
    c.update(batch=_log(rng, 1, 64), lo=0, hi=_log(rng, 1, 2000), new_hi=hi)
    if op == "load":
        c["batch"] = max(1, min(c["batch"], 67108864 // (hi * hk * c["dim"])))
    c["new_lo"] = min(hi, rng.choice([0, 1])) if hi > 1 else 1
    if op == "append":
        f = c["dim"]
        c.update(hq=hk * group, rotary=rng.choice([f, f, f // 2, min(f, 40), min(f, 22)]), axes=rng.randint(1, 4),
                 interleaved=rng.random() < 0.4)
    return c


# ---------------------------------------------------------------- what the sizes of a case are

def _spread(lo, hi, n):
    """n lengths over [lo, hi], the longest among them."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) if hi > lo else hi for i in range(n)]


def _sections(c):
    f = c["rotary"] // 2
    base = [f // c["axes"]] * c["axes"]
    base[0] += f - sum(base)
    return base


def _old(c):
    return _spread(c["lo"], c["hi"], c["batch"])[::-1]


def _new(c):
    return _spread(c["new_lo"], c["new_hi"], c["batch"])


def _starts(c):
    """First slots of what an append reads back: those of the blocks that it changes."""
    return [x // c["block"] * c["block"] if c["op"] == "append" else x for x in _old(c)]


def _back(c):
    """How many slots an append or a load reads back, by sequence."""
    return [x + y - z if y else 0 for x, y, z in zip(_old(c), _new(c), _starts(c))]


def _parents(c):
    """Groups of `beams` rows that take places among themselves; of every fifth group all end, where some have."""
    got = []
    for b in range(c["batch"]):
        g, i = divmod(b, c["beams"])
        n = min(c["beams"], c["batch"] - g * c["beams"])
        got.append(-1 if c["ended"] and g % 5 == 4 else g * c["beams"] + (i * i + g) % max(1, (n + 1) // 2))
    return got


def _fork_sizes(c):
    lens = _spread(c["lo"], c["hi"], c["batch"])
    held = [-(-n // c["page"]) for n in lens]
    return lens, held, max(1, -(-(max(lens) + c["room"]) // c["page"]))


def work(c):
    d = c.get("dim", 0)
    if c["op"] == "append":
        n, r = sum(_new(c)), sum(_back(c))
        blocks = sum(-(-x // c["block"]) for x in _back(c))
        return {"bytes": n * d * (4 * c["hq"] + 6 * c["hk"]) + 4 * c["axes"] * n + 8 * c["batch"] + r * c["hk"] * d * 6
                + blocks * c["hk"] * 24, "flops": 3 * n * (c["hq"] + c["hk"]) * c["rotary"] + 6 * n * c["hk"] * d + 2 * r * c["hk"] * d}
    if c["op"] == "load":
        r = sum(_back(c))
        return {"bytes": r * c["hk"] * d * 6 + r * c["hk"] * 8 // c["block"] + 8 * c["batch"], "flops": 2 * r * c["hk"] * d}
    if c["op"] == "decode":
        lens = _spread(c["lo"], c["hi"], c["batch"])
        seen = sum(n if c["window"] < 0 else min(n, c["window"] + 1) for n in lens)
        return {"bytes": max(1, seen * c["hk"] * 2 * d + seen * c["hk"] * 8 // c["block"]
                             + c["batch"] * c["hq"] * (4 * d + 4) + 4 * c["batch"]), "flops": 4 * seen * c["hq"] * d}
    if c["op"] == "fork":
        _, held, width = _fork_sizes(c)
        pages = sum(held) + c["spare"]
        return {"bytes": 8 * c["batch"] * width + 8 * pages + 16 * c["batch"], "flops": pages + c["batch"] * width}
    size = 1 if c["kind"] else 2
    scales = 8 * c["page"] // c["block"] * c["hk"] if c["kind"] else 0
    return {"bytes": 2 * c["pairs"] * (2 * c["page"] * c["hk"] * d * size + scales) + 8 * c["pairs"], "flops": 0}


# ---------------------------------------------------------------- inputs

def _codes(shape, kind, g):
    """Codes of normally distributed values."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    if kind == "int8":
        return t.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    return t.mul_(100.0).clamp_(-448, 448).to(torch.float8_e4m3fn) if kind else t


def _pages(c, pages, g):
    """Pages of keys and values in the case's type and, in 8 bits, their factors (powers of two)."""
    shape = (pages, c["hk"], c["page"], c["dim"]) if c["heads_first"] else (pages, c["page"], c["hk"], c["dim"])
    made = []
    for _ in range(2):
        t = _codes(shape, c["kind"], g)
        t = t if c["kind"] else t.to(DT[c["dtype"]])
        made.append(t.transpose(1, 2) if c["heads_first"] else t)
    for _ in range(2):
        e = torch.randint(-7, -4, (pages, c["page"] // c["block"], c["hk"]), generator=g, device=DEV)
        made.append(torch.exp2(e.float()) if c["kind"] else None)
    return made


def _cache(c, capacity, g):
    """Pages in a random order: {"kc", "vc", "ks", "vs", "table"}."""
    per = max(1, -(-capacity // c["page"]))
    pages = c["batch"] * per + 3
    kc, vc, ks, vs = _pages(c, pages, g)
    table = torch.randperm(pages, generator=g, device=DEV)[:c["batch"] * per]
    return {"kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table.to(torch.int32).view(c["batch"], per)}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}

    def rand(*shape):
        # heads differ in size, and a few tokens stand out
        t = torch.randn(*shape, generator=g, device=DEV)
        t *= 1.0 + 7.0 * (torch.rand(shape[0], shape[1], 1, generator=g, device=DEV) < 0.02)
        return t.to(DT[c["dtype"]])

    if c["op"] in ("append", "load"):
        old, new = _old(c), _new(c)
        s["cap"] = max(1, max(x + y for x, y in zip(old, new)))
        s.update(_cache(c, s["cap"], g))
        s["seqlens"], s["cu"] = _ints(old), _ints(_offsets(new))
        s["starts"], s["cu_back"], s["back"] = _ints(_starts(c)), _ints(_offsets(_back(c))), sum(_back(c))
        n = sum(new)
        if c["op"] == "append":
            s["q"], s["k"], s["v"] = rand(n, c["hq"], c["dim"]), rand(n, c["hk"], c["dim"]), rand(n, c["hk"], c["dim"])
            f = c["rotary"] // 2
            s["inv"] = (1.0 / (10000.0 ** (torch.arange(f, dtype=torch.float64) / f))).to(device=DEV, dtype=torch.float32)
            s["pos"] = torch.randint(0, 100000, (c["axes"], n), generator=g, device=DEV, dtype=torch.int32)
    elif c["op"] == "decode":
        lens = _spread(c["lo"], c["hi"], c["batch"])
        s["cap"] = max(1, max(lens))
        s.update(_cache(c, s["cap"], g))
        s["seqlens"] = _ints(lens)
        s["q"] = rand(c["batch"], c["hq"], c["dim"])
    elif c["op"] == "fork":
        lens, held, width = _fork_sizes(c)
        pages = sum(held) + c["spare"]
        at = torch.randperm(pages, generator=g, device=DEV)
        of = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), torch.tensor(held, device=DEV))
        within = torch.arange(len(of), device=DEV) - torch.tensor(_offsets(held)[:-1], device=DEV)[of]
        s["table"] = torch.full((c["batch"], width), -1, dtype=torch.int32, device=DEV)
        s["table"][of, within] = at[:len(of)].to(torch.int32)
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        s["refs"][at[:len(of)]] = 1
        # of each group a few pages belong to all rows, as after an earlier fork
        first = torch.arange(c["batch"], device=DEV) // c["beams"] * c["beams"]
        same = torch.tensor(lens, device=DEV).div(c["page"], rounding_mode="floor")
        for i in range(min(3, width)):
            both = (same > i) & (same[first] > i) & (first != torch.arange(c["batch"], device=DEV))
            rows = both.nonzero().view(-1)
            gone, kept = s["table"][rows, i].long(), s["table"][first[rows], i].long()
            s["table"][rows, i] = kept.to(torch.int32)
            s["refs"].index_add_(0, kept, torch.ones_like(kept, dtype=torch.int32))
            s["refs"][gone] = 0
        s["seqlens"], s["parents"] = _ints(lens), _ints(_parents(c))
        s["room"] = _ints([c["room"]] * c["batch"])
        s["table_out"], s["seqlens_out"] = torch.empty_like(s["table"]), torch.empty_like(s["seqlens"])
        s["refs_out"] = torch.empty_like(s["refs"])
        most = c["batch"] if c["share"] else c["batch"] * width
        s["copies"] = torch.full((most, 2), -1, dtype=torch.int32, device=DEV)
        s["counts"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    else:
        s["kc"], s["vc"], s["ks"], s["vs"] = _pages(c, c["pages"], g)
        at = torch.randperm(c["pages"], generator=g, device=DEV)[:2 * c["pairs"]].to(torch.int32)
        s["pairs"] = at.view(c["pairs"], 2).contiguous()
    return s


# ---------------------------------------------------------------- one pass, in plain operations

def _turned(x, pos, inv, c):
    """x [tokens, heads, dim] rotated by the positions of its tokens, in 64 bits: codes turn over at borders."""
    f = c["rotary"] // 2
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(_sections(c), device=DEV))
    angle = pos.double().movedim(0, -1)[..., axis] * inv.double()
    cos, sin = angle.cos().unsqueeze(-2), angle.sin().unsqueeze(-2)
    y = x.double()
    if c["interleaved"]:
        a, b = y[..., 0:2 * f:2], y[..., 1:2 * f:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :f], y[..., f:2 * f]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., 2 * f:]], -1)


def _to_codes(x, kind):
    x = x.clamp(-TOP[kind], TOP[kind])
    return x.round().to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn)


def _put(pages, page, within, codes):
    """pages[page, within] = codes, byte by byte."""
    pages.view(torch.uint8)[page, within] = codes.view(torch.uint8)


def _taken(pages, page, within):
    return pages.view(torch.uint8)[page, within].view(pages.dtype)


def _factor(top, kind):
    """The smallest power of two that `top` is at most TOP times of."""
    m, e = torch.frexp(top / TOP[kind])
    e = torch.where(m == 0.5, e - 1, e).double()
    return torch.exp2(torch.where(top > 0, e, torch.full_like(e, -60.0)).clamp(-60, 60))


def _append(s):
    c = s["case"]
    old, cu, table, page, block = s["seqlens"].long(), s["cu"].long(), s["table"].long(), c["page"], c["block"]
    t = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    slot = old[seq] + t - cu[seq]
    at, within = table[seq, slot // page], slot % page
    # the slots that the first block of each sequence holds already
    j = old[:, None] // block * block + torch.arange(block, device=DEV)
    held = (j < old[:, None]) & (cu[1:] > cu[:-1])[:, None]
    hp, hw = table.gather(1, (j // page).clamp(max=table.shape[1] - 1))[held], (j % page)[held]
    for x, pages, scales in ((_turned(s["k"], s["pos"], s["inv"], c), s["kc"], s["ks"]), (s["v"].double(), s["vc"], s["vs"])):
        row = at * (page // block) + within // block
        top = torch.zeros(scales.shape[0] * scales.shape[1], c["hk"], dtype=torch.float64, device=DEV)
        top.scatter_reduce_(0, row[:, None].expand(-1, c["hk"]), x.abs().amax(-1), "amax")
        base = torch.zeros(len(top), 1, dtype=torch.bool, device=DEV)
        base[hp * (page // block) + hw // block] = True
        was = scales.reshape(-1, c["hk"]).double()
        now = torch.maximum(_factor(top, c["kind"]), torch.where(base, was, torch.zeros_like(was)))
        touched = torch.zeros_like(base)
        touched[row] = True
        now = torch.where(touched, now, was)
        hr = hp * (page // block) + hw // block
        before = _taken(pages, hp, hw).double() * (was[hr] / now[hr])[..., None]
        _put(pages, hp, hw, _to_codes(before, c["kind"]))
        _put(pages, at, within, _to_codes(x / now[row][..., None], c["kind"]))
        scales.copy_(now.view(scales.shape))
    k, v = _load(s)
    return {"q": _turned(s["q"], s["pos"], s["inv"], c).to(DT[c["dtype"]]), "k": k, "v": v, "k_scale": s["ks"], "v_scale": s["vs"]}


def _load(s):
    c = s["case"]
    t = torch.arange(s["back"], device=DEV)
    cu = s["cu_back"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    slot = s["starts"].long()[seq] + t - cu[seq]
    at, within = s["table"].long()[seq, slot // c["page"]], slot % c["page"]
    return [(_taken(p, at, within).float() * f[at, within // c["block"]][..., None]).to(DT[c["dtype"]])
            for p, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]


def _decode(s):
    c = s["case"]
    b, cap, group = c["batch"], s["cap"], c["hq"] // c["hk"]
    j = torch.arange(cap, device=DEV)
    n = s["seqlens"].long()
    page, within = s["table"].long()[:, j // c["page"]], j % c["page"]
    k, v = (_taken(p, page, within).float() * f[page, within // c["block"]][..., None]
            for p, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))  # [batch, cap, hk, dim]
    q = s["q"].float().view(b, c["hk"], group, c["dim"])
    x = torch.einsum("bhgd,bjhd->bhgj", q, k) * c["dim"] ** -0.5
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    live = j < n[:, None]
    if c["window"] >= 0:
        live = live & (j >= n[:, None] - 1 - c["window"])
    x = x.masked_fill(~live[:, None, None], -INF)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -INF, top, torch.zeros_like(top))
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p = p / torch.where(some, total, torch.ones_like(total))
    out = torch.einsum("bhgj,bjhd->bhgd", p, v).reshape(b, c["hq"], c["dim"]).to(DT[c["dtype"]])
    lse = torch.where(some, top + total.log(), torch.full_like(top, INF)).reshape(b, c["hq"])
    return {"out": out, "lse": lse}


def _fork(s):
    c, page = s["case"], s["case"]["page"]
    table, n0, refs = s["table"].long(), s["seqlens"].long(), s["refs"].long()
    rows, width = table.shape
    b, i = torch.arange(rows, device=DEV), torch.arange(width, device=DEV)
    live, src = s["parents"].long() >= 0, s["parents"].long().clamp(min=0)
    # the first row of each parent goes on with its pages, the others share the full ones
    who = torch.full((rows,), rows, device=DEV)
    who.scatter_reduce_(0, src, torch.where(live, b, torch.full_like(b, rows)), "amin")
    heir = (live & (who[src] == b))[:, None]
    n = torch.where(live, n0[src], torch.zeros_like(n0))[:, None]
    used, need = (n + page - 1) // page, (n + s["room"].long()[:, None] + page - 1) // page
    old = table[src]
    shared = live[:, None] & ~heir & (i < n // page) & c["share"]
    new = torch.where(heir | shared, old, torch.full_like(old, -1))
    copied = live[:, None] & ~heir & ~shared & (i < used)
    fresh = copied | (live[:, None] & (i >= used) & (i < need) & (new < 0))
    left = torch.where((who == rows)[:, None] & (table >= 0), table, torch.full_like(table, -1))
    for pages, sign in ((left, -1), (torch.where(shared, old, torch.full_like(old, -1)), 1)):
        pages = pages.reshape(-1)
        refs.index_add_(0, pages.clamp(min=0), torch.where(pages >= 0, sign, 0))
    free = (refs != 0).to(torch.uint8).sort(stable=True).indices  # the free pages first, in order
    rank = fresh.view(-1).cumsum(0).view(rows, width) - 1
    got = fresh & (rank < (refs == 0).sum())
    taken = torch.where(got, free[rank.clamp(0, len(free) - 1)], torch.full_like(rank, -1))
    new = torch.where(fresh, taken, new)
    refs.index_add_(0, taken.clamp(min=0).view(-1), got.long().view(-1))
    made = copied & got
    place = made.view(-1).cumsum(0).view(rows, width) - 1
    most = len(s["copies"])
    pairs = torch.cat([s["copies"].long(), torch.zeros(1, 2, dtype=torch.long, device=DEV)])
    pairs[torch.where(made, place, torch.full_like(place, most)).view(-1)] = torch.stack([old, new], -1).view(-1, 2)
    s["copies"].copy_(pairs[:most])
    s["counts"].copy_(torch.stack([made.sum(), (refs == 0).sum()]))
    s["table_out"].copy_(new)
    s["seqlens_out"].copy_(n[:, 0])
    s["refs_out"].copy_(refs)
    return {n: s[n] for n in ("table_out", "seqlens_out", "refs_out", "copies", "counts")}


def _copy(s):
    src, dst = s["pairs"].long().unbind(1)
    for p in (s["kc"], s["vc"]):
        p = p.view(torch.uint8)
        p[dst] = p[src]
    got = {"k_cache": s["kc"], "v_cache": s["vc"]}
    if s["ks"] is not None:
        s["ks"][dst], s["vs"][dst] = s["ks"][src], s["vs"][src]
        got.update(k_scale=s["ks"], v_scale=s["vs"])
    return got


def _own(s):
    import attention_backward_bwd_gb300 as ab
    c = s["case"]
    if c["op"] == "append":
        q = ab.attn_cache_append8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["seqlens"],
                                  cu_seqlens=s["cu"], q=s["q"], positions=s["pos"], inv_freq=s["inv"],
                                  sections=_sections(c), interleaved=c["interleaved"])
        k, v = ab.attn_cache_load8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["starts"], s["cu_back"], s["back"],
                                   dtype=DT[c["dtype"]])
        return {"q": q, "k": k, "v": v, "k_scale": s["ks"], "v_scale": s["vs"]}
    if c["op"] == "load":
        return ab.attn_cache_load8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["starts"], s["cu_back"], s["back"],
                                   dtype=DT[c["dtype"]])
    if c["op"] == "decode":
        out, lse = ab.attn_decode8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["seqlens"],
                                   max_seqlen=s["cap"], window=(c["window"], -1), softcap=c["cap"])
        return {"out": out, "lse": lse}
    if c["op"] == "fork":
        ab.attn_cache_fork(s["table"], s["seqlens"], s["refs"], c["page"], parents=s["parents"], room=s["room"],
                           share=c["share"], table_out=s["table_out"], seqlens_out=s["seqlens_out"],
                           refs_out=s["refs_out"], copies=s["copies"], counts=s["counts"])
        return {n: s[n] for n in ("table_out", "seqlens_out", "refs_out", "copies", "counts")}
    ab.attn_cache_copy(s["kc"], s["vc"], s["pairs"], k_scale=s["ks"], v_scale=s["vs"])
    got = {"k_cache": s["kc"], "v_cache": s["vc"]}
    if s["ks"] is not None:
        got.update(k_scale=s["ks"], v_scale=s["vs"])
    return got


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "load": _load, "decode": _decode, "fork": _fork, "copy": _copy}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _turned64(x, pos, inv, c):
    """As complex numbers: each pair times e^(i angle)."""
    f, sec = c["rotary"] // 2, _sections(c)
    x = x.double()
    angle = torch.empty(*pos.shape[1:], f, dtype=torch.float64, device=DEV)
    for a in range(len(sec)):
        at, end = sum(sec[:a]), sum(sec[:a + 1])
        angle[..., at:end] = pos[a].double()[..., None] * inv[at:end].double()
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(-2)
    pair = (slice(0, 2 * f, 2), slice(1, 2 * f, 2)) if c["interleaved"] else (slice(0, f), slice(f, 2 * f))
    z = torch.complex(x[..., pair[0]].contiguous(), x[..., pair[1]].contiguous()) * turn
    x[..., pair[0]], x[..., pair[1]] = z.real, z.imag
    return x


def _held64(s, pages, scales, b, at, end):
    """Values of slots [at, end) of sequence b, slot by slot of the block table."""
    c = s["case"]
    j = torch.arange(at, end, device=DEV)
    rows = s["table"][b].long()[j // c["page"]]
    f = scales[rows, j % c["page"] // c["block"]].double()
    return pages.view(torch.uint8)[rows, j % c["page"]].view(pages.dtype).double() * f[..., None]


def _rounded64(x, kind):
    """Values with the nearest code, ties to the even one."""
    if kind == "int8":
        return x.round().clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(torch.exp2(e) > x.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def exact(case, seed):
    if case["op"] in ("fork", "copy"):
        return None
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "decode":
        g = c["hq"] // c["hk"]
        out = torch.zeros(c["batch"], c["hq"], c["dim"], dtype=torch.float64, device=DEV)
        lse = torch.full((c["batch"], c["hq"]), INF, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["seqlens"].tolist()):
            at = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
            if n == 0:
                continue
            for h in range(c["hk"]):
                k, v = (_held64(s, p[:, :, h:h + 1], f[:, :, h:h + 1], b, at, n)[:, 0]
                        for p, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
                x = s["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(c["dim"])
                x = c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] > 0 else x
                lse[b, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
                out[b, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
        return {"out": out, "lse": lse}
    at, cu = s["starts"].tolist(), s["cu_back"].tolist()
    if c["op"] == "load":
        both = [torch.cat([_held64(s, p, f, b, at[b], at[b] + cu[b + 1] - cu[b]) for b in range(c["batch"])])
                for p, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]
        return both
    got = {"q": _turned64(s["q"], s["pos"], s["inv"], c)}
    first, new, block = s["cu"].tolist(), _new(c), c["block"]
    for name, x, pages, scales in (("k", _turned64(s["k"], s["pos"], s["inv"], c), s["kc"], s["ks"]),
                                   ("v", s["v"].double(), s["vc"], s["vs"])):
        after, values = scales.double(), []
        for b, old in enumerate(s["seqlens"].tolist()):
            if new[b] == 0:
                continue
            rows = torch.cat([_held64(s, pages, scales, b, at[b], old), x[first[b]:first[b + 1]]])
            n = len(rows)
            count = -(-n // block)
            full = torch.zeros(count * block, c["hk"], c["dim"], dtype=torch.float64, device=DEV)
            full[:n] = rows
            fresh = full.clone()
            fresh[:old - at[b]] = 0.0
            top = fresh.view(count, block, c["hk"], c["dim"]).abs().amax((1, 3)) / TOP[c["kind"]]
            f = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -60))))
            f = torch.where(f / 2 >= top, f / 2, f)  # log2 next to a whole number
            j = at[b] + block * torch.arange(count, device=DEV)
            page, within = s["table"][b].long()[j // c["page"]], j % c["page"] // block
            f = torch.where(((j < old)[:, None]) & (scales[page, within].double() > f), scales[page, within].double(), f)
            after[page, within] = f
            f = f.repeat_interleave(block, 0)[:n, :, None]
            values.append(_rounded64(rows / f, c["kind"]) * f)
        got[name], got[name + "_scale"] = torch.cat(values), after
    return got
