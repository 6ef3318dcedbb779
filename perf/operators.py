"""Cases and plain forms of the serving operators: rotary positions, the paged key-value cache's
append, single-token attention over the cache and eviction by accumulated attention weight.

``run`` takes what ``prepare`` made and makes one pass through one operator: in plain torch
operations where ``own`` is false, through the package's entry points where it is true.
``exact`` computes the same outputs in 64 bits, apart from the plain form.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
INF = float("inf")


def listed():
    return [
        # the training workload's q and k rotated before the forward; video positions (time, height, width)
        {"name": "rope_train", "op": "rope", "dtype": "bf16", "batch": 2, "tokens": 8192, "hq": 32, "hk": 8,
         "dim": 128, "rotary": 128, "axes": 3, "interleaved": False, "inverse": False, "far": 40000},
        # gradients of packed odd-length text, rotated back: neighbouring pairs, part of the head rotated
        {"name": "rope_grad_packed", "op": "rope", "dtype": "fp16", "batch": 0, "tokens": 5077, "hq": 16, "hk": 16,
         "dim": 96, "rotary": 64, "axes": 1, "interleaved": True, "inverse": True, "far": 1000000},
        # a decode step of a batch: one token a sequence, q rotated in the same call
        {"name": "append_step", "op": "append", "dtype": "bf16", "batch": 64, "lo": 100, "hi": 2000, "new_lo": 1,
         "new_hi": 1, "hq": 32, "hk": 8, "dim": 128, "rotary": 128, "axes": 1, "interleaved": False, "page": 64,
         "heads_first": False},
        # ragged prompts entering the cache, with positions of images among the text
        {"name": "append_prompts", "op": "append", "dtype": "fp16", "batch": 16, "lo": 0, "hi": 300, "new_lo": 128,
         "new_hi": 2048, "hq": 16, "hk": 16, "dim": 128, "rotary": 96, "axes": 2, "interleaved": True, "page": 16,
         "heads_first": True},
        # one short chat on small heads: latency alone
        {"name": "decode_smallest", "op": "decode", "dtype": "fp16", "batch": 1, "lo": 128, "hi": 128, "hq": 2, "hk": 2,
         "dim": 64, "page": 16, "window": -1, "cap": 0.0, "weights": False, "heads_first": False},
        # a serving batch of ragged chats
        {"name": "decode_batch", "op": "decode", "dtype": "bf16", "batch": 32, "lo": 128, "hi": 8192, "hq": 32,
         "hk": 8, "dim": 128, "page": 64, "window": -1, "cap": 0.0, "weights": False, "heads_first": False},
        # one user with a very long document: the length has to be split
        {"name": "decode_long", "op": "decode", "dtype": "bf16", "batch": 1, "lo": 131071, "hi": 131071, "hq": 32,
         "hk": 8, "dim": 128, "page": 128, "window": -1, "cap": 0.0, "weights": False, "heads_first": True},
        # the largest batch of long chats
        {"name": "decode_largest", "op": "decode", "dtype": "bf16", "batch": 64, "lo": 4096, "hi": 16384, "hq": 32,
         "hk": 8, "dim": 128, "page": 16, "window": -1, "cap": 0.0, "weights": False, "heads_first": False},
        # wide heads without sharing, a sliding window and a logit cap, pages of an odd size
        {"name": "decode_window_cap", "op": "decode", "dtype": "fp16", "batch": 9, "lo": 1, "hi": 4096, "hq": 16,
         "hk": 16, "dim": 256, "page": 48, "window": 1024, "cap": 30.0, "weights": False, "heads_first": False},
        # decode that also gathers each key's attention weight
        {"name": "decode_weights", "op": "decode", "dtype": "bf16", "batch": 8, "lo": 1000, "hi": 16384, "hq": 32,
         "hk": 8, "dim": 128, "page": 32, "window": -1, "cap": 0.0, "weights": True, "heads_first": False},
        # prompts cut down to the cache's budget
        {"name": "evict_prompts", "op": "evict", "dtype": "bf16", "batch": 4, "lo": 5000, "hi": 16000, "hk": 8,
         "dim": 128, "page": 64, "budget": 1024, "recent": 256, "settled": False, "heads_first": False},
        # the steady state of a batch: a few new tokens each, back to the budget
        {"name": "evict_steady", "op": "evict", "dtype": "fp16", "batch": 64, "lo": 1025, "hi": 1088, "hk": 16,
         "dim": 64, "page": 16, "budget": 1024, "recent": 128, "settled": True, "heads_first": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    c = {"op": op, "dtype": rng.choice(["fp16", "bf16"])}
    hk = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16, 20]) if hk <= 8 else rng.choice([1, 2])
    dim = rng.choice([64, 72, 80, 96, 112, 128, 192, 256])
    rotary = {"dim": dim, "rotary": rng.choice([dim, dim, dim // 2 // 2 * 2, 40, 22]), "axes": rng.randint(1, 4),
              "interleaved": rng.random() < 0.4}
    cache = {"page": rng.choice([1, 8, 16, 16, 32, 48, 64, 100, 128, 256]), "heads_first": rng.random() < 0.5}
    if op == "rope":
        c.update(batch=rng.choice([0, 0, 1, 2, 3]), tokens=_log(rng, 1, 8192), hq=hk * group, hk=hk, **rotary,
                 inverse=rng.random() < 0.5, far=_log(rng, 100, 2000000))
        c["tokens"] = max(1, min(c["tokens"], 16384 * 40 * 128 // (max(1, c["batch"]) * (hk * group + hk) * dim)))
    elif op == "append":
        hi = rng.choice([1, 1, _log(rng, 1, 2048)])
        c.update(batch=_log(rng, 1, 64), lo=0, hi=_log(rng, 1, 2000), new_lo=min(hi, rng.choice([0, 1])) if hi > 1 else 1,
                 new_hi=hi, hq=hk * group, hk=hk, **rotary, **cache)
    elif op == "decode":
        batch, hi = _log(rng, 1, 128), _log(rng, 1, 131072)
        hi = max(1, min(hi, 40000000 // (batch * hk * dim // 8)))
        c.update(batch=batch, lo=rng.choice([0, 1, max(1, hi // 2)]) if batch > 1 else max(1, hi // 2), hi=hi, hq=hk * group,
                 hk=hk, dim=dim, window=rng.choice([-1, -1, _log(rng, 1, 4096)]), cap=rng.choice([0.0, 0.0, 20.0]),
                 weights=rng.random() < 0.4, **cache)
    else:
        batch, budget = _log(rng, 1, 64), _log(rng, 64, 2048)
        hi = max(budget + 1, min(_log(rng, budget + 1, 32768), 40000000 // (batch * hk * dim // 4)))
        c.update(batch=batch, lo=rng.choice([1, budget + 1, max(1, hi // 2)]), hi=hi, hk=hk, dim=dim, budget=budget,
                 recent=rng.choice([0, 1, budget // 4, budget // 2]), settled=rng.random() < 0.5, **cache)
        c["lo"] = min(c["lo"], hi)
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


def _tokens(c):
    return max(1, c["batch"]) * c["tokens"]


def _new(c):
    return _spread(c["new_lo"], c["new_hi"], c["batch"])


def work(c):
    d, e = c["dim"], 2
    if c["op"] == "rope":
        n = _tokens(c) * (c["hq"] + c["hk"])
        return {"bytes": 2 * n * d * e + 4 * c["axes"] * _tokens(c), "flops": 3 * n * c["rotary"]}
    if c["op"] == "append":
        n = sum(_new(c))
        return {"bytes": n * (2 * c["hq"] + 4 * c["hk"]) * d * e + 4 * c["axes"] * n + 8 * c["batch"],
                "flops": 3 * n * (c["hq"] + c["hk"]) * c["rotary"]}
    lens = _spread(c["lo"], c["hi"], c["batch"])
    if c["op"] == "decode":
        seen = sum(n if c["window"] < 0 else min(n, c["window"] + 1) for n in lens)
        b = seen * c["hk"] * d * 2 * e + 2 * c["batch"] * c["hq"] * d * e + 4 * c["batch"] * (c["hq"] + 1)
        return {"bytes": b + (8 * sum(lens) * c["hk"] if c["weights"] else 0), "flops": 4 * seen * c["hq"] * d}
    moved = slots = 0
    for n in lens:
        slots += n
        if n > c["budget"]:
            above, r = n - c["budget"], c["recent"]
            fresh = min(above, r)  # protected slots above the budget; the rest competes by weight
            moved += fresh + (above - fresh) * (c["budget"] - r) / max(1, n - r)
    return {"bytes": c["hk"] * (slots * 16 + moved * d * 4 * e), "flops": c["hk"] * slots}


# ---------------------------------------------------------------- inputs

def _cache(c, capacity, g):
    """Pages of random values in a random order: (k_cache, v_cache, block_table)."""
    per = max(1, -(-capacity // c["page"]))
    pages, dt = c["batch"] * per + 3, DT[c["dtype"]]
    shape = (pages, c["hk"], c["page"], c["dim"]) if c["heads_first"] else (pages, c["page"], c["hk"], c["dim"])
    made = []
    for _ in range(2):
        t = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)
        made.append(t.transpose(1, 2) if c["heads_first"] else t)
    table = torch.randperm(pages, generator=g, device=DEV)[:c["batch"] * per]
    return made[0], made[1], table.to(torch.int32).view(c["batch"], per)


def _rotary(c, tokens, far, g):
    f = c["rotary"] // 2
    inv = 1.0 / (10000.0 ** (torch.arange(f, dtype=torch.float64) / f))
    pos = torch.randint(0, far, (c["axes"], tokens), generator=g, device=DEV, dtype=torch.int32)
    return pos, inv.to(device=DEV, dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(dt)

    s = {"case": c}
    if c["op"] == "rope":
        lead = (c["tokens"],) if c["batch"] == 0 else (c["batch"], c["tokens"])
        s["q"], s["k"] = rand(*lead, c["hq"], c["dim"]), rand(*lead, c["hk"], c["dim"])
        pos, s["inv"] = _rotary(c, _tokens(c), c["far"], g)
        s["pos"] = pos.view(c["axes"], *lead)
    elif c["op"] == "append":
        old, new = _spread(c["lo"], c["hi"], c["batch"])[::-1], _new(c)
        n = sum(new)
        s["seqlens"], s["seen"] = _ints(old), _ints([x + 7 for x in old])
        s["cu"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
        s["cap"] = max(x + y for x, y in zip(old, new))
        s["kc"], s["vc"], s["table"] = _cache(c, s["cap"], g)
        s["q"], s["k"], s["v"] = rand(n, c["hq"], c["dim"]), rand(n, c["hk"], c["dim"]), rand(n, c["hk"], c["dim"])
        s["pos"], s["inv"] = _rotary(c, n, 100000, g)
        s["slots"] = torch.full((c["batch"], c["hk"], s["cap"]), -1, dtype=torch.int32, device=DEV)
    else:
        lens = _spread(c["lo"], c["hi"], c["batch"])
        s["cap"] = max(1, max(lens))
        s["seqlens"] = _ints(lens)
        s["kc"], s["vc"], s["table"] = _cache(c, s["cap"], g)
        if c["op"] == "decode":
            s["q"] = rand(c["batch"], c["hq"], c["dim"])
        # attention weights gathered so far: a few keys hold most of them
        s["w"] = torch.randn(c["batch"], c["hk"], s["cap"], generator=g, device=DEV).mul_(2.0).exp_()
        s["w_out"] = torch.zeros_like(s["w"])
        if c["op"] == "evict":
            slot = torch.arange(s["cap"], dtype=torch.int32, device=DEV).expand(c["batch"], c["hk"], s["cap"])
            if c["settled"]:  # evicted before: the first slots hold older tokens in any order
                old = min(c["budget"], s["cap"])
                mix = torch.rand(c["batch"], c["hk"], old, generator=g, device=DEV).argsort(-1).to(torch.int32)
                slot = torch.cat([mix, slot[..., old:]], -1)
            s["slots"] = slot.contiguous()
            s["slots_out"] = torch.full_like(s["slots"], -1)
            s["seen"] = s["seqlens"].clone()
    return s


# ---------------------------------------------------------------- one pass

def _turned(x, pos, inv, c, inverse=False):
    """x [..., heads, dim] rotated by the positions of its tokens, in 32 bits, rounded once."""
    f = c["rotary"] // 2
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(_sections(c), device=DEV))
    angle = pos.double().movedim(0, -1)[..., axis] * inv.double()
    cos, sin = angle.cos().float().unsqueeze(-2), angle.sin().float().unsqueeze(-2)
    sin = -sin if inverse else sin
    y = x.float()
    if c["interleaved"]:
        a, b = y[..., 0:2 * f:2], y[..., 1:2 * f:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :f], y[..., f:2 * f]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., 2 * f:]], -1).to(x.dtype)


def _append(s):
    c = s["case"]
    t = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    i = t - s["cu"].long()[seq]
    slot = s["seqlens"].long()[seq] + i
    page = s["table"].long()[seq, slot // c["page"]]
    s["kc"][page, slot % c["page"]] = _turned(s["k"], s["pos"], s["inv"], c)
    s["vc"][page, slot % c["page"]] = s["v"]
    s["slots"][seq, :, slot] = (s["seen"].long()[seq] + i).to(torch.int32).unsqueeze(-1).expand(-1, c["hk"])
    return {"q": _turned(s["q"], s["pos"], s["inv"], c), "k_cache": s["kc"], "v_cache": s["vc"], "slots": s["slots"]}


def _decode(s):
    c = s["case"]
    b, cap, group = c["batch"], s["cap"], c["hq"] // c["hk"]
    j = torch.arange(cap, device=DEV)
    n = s["seqlens"].long()
    page, within = s["table"].long()[:, j // c["page"]], j % c["page"]
    k, v = s["kc"][page, within].float(), s["vc"][page, within].float()  # [batch, cap, hk, dim]
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
    got = {"out": out, "lse": lse}
    if c["weights"]:
        inside = (j < n[:, None])[:, None]
        s["w_out"].copy_(torch.where(inside, s["w"] + p.sum(2), s["w_out"]))
        got["weights"] = s["w_out"]
    return got


def _evict(s):
    c = s["case"]
    cap, budget = s["cap"], c["budget"]
    n = s["seqlens"].long()[:, None, None]
    j = torch.arange(cap, device=DEV)
    inside = (j < n).expand_as(s["w"])
    held = inside & (s["slots"].long() >= s["seen"].long()[:, None, None] - c["recent"])
    rank = torch.where(held, torch.full_like(s["w"], INF), s["w"])
    rank = torch.where(inside, rank, torch.full_like(s["w"], -INF))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.zeros_like(inside).scatter_(-1, order, True) & inside
    out = torch.clamp(n, max=budget)
    hole, mover = (~kept) & inside & (j < budget), kept & (j >= budget)
    to, of = hole.nonzero(), mover.nonzero()  # the same (sequence, head) at the same place, slots ascending
    source, held_in = torch.where(inside, s["w"], s["w_out"]), torch.where(inside, s["slots"], s["slots_out"])
    w, pos = source.clone(), held_in.clone()
    w[tuple(to.T)] = source[tuple(of.T)]
    pos[tuple(to.T)] = held_in[tuple(of.T)]
    gone = inside & (j >= out)
    s["w_out"].copy_(w.masked_fill(gone, 0.0))
    s["slots_out"].copy_(pos.masked_fill(gone, -1))
    seq, head = to[:, 0], to[:, 1]
    table = s["table"].long()
    for pages in (s["kc"], s["vc"]):
        rows = pages[table[seq, of[:, 2] // c["page"]], of[:, 2] % c["page"], head]
        pages[table[seq, to[:, 2] // c["page"]], to[:, 2] % c["page"], head] = rows
    return {"k_cache": s["kc"], "v_cache": s["vc"], "seqlens": out.view(-1).to(torch.int32), "weights": s["w_out"],
            "slots": s["slots_out"]}


def _own(s):
    import attention_backward_bwd_gb300 as ab
    c = s["case"]
    if c["op"] == "rope":
        q, k = ab.attn_rope(s["q"], s["k"], s["pos"], s["inv"], sections=_sections(c), interleaved=c["interleaved"],
                            inverse=c["inverse"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        q = ab.attn_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["seqlens"], cu_seqlens=s["cu"], q=s["q"],
                                 positions=s["pos"], inv_freq=s["inv"], sections=_sections(c),
                                 interleaved=c["interleaved"], slot_positions=s["slots"], seen=s["seen"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"], "slots": s["slots"]}
    if c["op"] == "decode":
        out, lse = ab.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["seqlens"], max_seqlen=s["cap"],
                                  window=(c["window"], -1), softcap=c["cap"], weights=s["w"] if c["weights"] else None,
                                  weights_out=s["w_out"] if c["weights"] else None)
        got = {"out": out, "lse": lse}
        if c["weights"]:
            got["weights"] = s["w_out"]
        return got
    lens, w, slots = ab.attn_cache_evict(s["kc"], s["vc"], s["table"], s["seqlens"], s["w"], c["budget"],
                                         recent=c["recent"], slot_positions=s["slots"], seen=s["seen"],
                                         max_seqlen=s["cap"], weights_out=s["w_out"], positions_out=s["slots_out"])
    return {"k_cache": s["kc"], "v_cache": s["vc"], "seqlens": lens, "weights": w, "slots": slots}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "rope":
        return {n: _turned(state[n], state["pos"], state["inv"], c, c["inverse"]) for n in ("q", "k")}
    return {"append": _append, "decode": _decode, "evict": _evict}[c["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _turned64(x, pos, inv, c, sign):
    """As complex numbers: each pair times e^(i angle)."""
    f, sec = c["rotary"] // 2, _sections(c)
    x = x.double()
    first = sum(sec[:1])
    angle = torch.empty(*pos.shape[1:], f, dtype=torch.float64, device=DEV)
    angle[..., :first] = pos[0].double()[..., None] * inv[:first].double()
    for a in range(1, len(sec)):
        at, end = sum(sec[:a]), sum(sec[:a + 1])
        angle[..., at:end] = pos[a].double()[..., None] * inv[at:end].double()
    turn = torch.polar(torch.ones_like(angle), sign * angle).unsqueeze(-2)
    pair = slice(0, 2 * f, 2), slice(1, 2 * f, 2)
    if not c["interleaved"]:
        pair = slice(0, f), slice(f, 2 * f)
    z = torch.complex(x[..., pair[0]].contiguous(), x[..., pair[1]].contiguous()) * turn
    x[..., pair[0]], x[..., pair[1]] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        sign = -1.0 if c["inverse"] else 1.0
        return {n: _turned64(s[n].clone(), s["pos"], s["inv"], c, sign) for n in ("q", "k")}
    table, page = s["table"].tolist(), c["page"]
    lens = s["seqlens"].tolist()
    if c["op"] == "append":
        q, k = (_turned64(s[n].clone(), s["pos"], s["inv"], c, 1.0) for n in ("q", "k"))
        kc, vc, cu = s["kc"].double(), s["vc"].double(), s["cu"].tolist()
        for b, old in enumerate(lens):
            at = cu[b]
            while at < cu[b + 1]:  # page by page
                slot = old + at - cu[b]
                m = min(page - slot % page, cu[b + 1] - at)
                p, o = table[b][slot // page], slot % page
                kc[p, o:o + m], vc[p, o:o + m] = k[at:at + m], s["v"][at:at + m].double()
                at += m
        return {"q": q, "k_cache": kc, "v_cache": vc, "slots": None}
    if c["op"] == "decode":
        g = c["hq"] // c["hk"]
        out = torch.zeros(c["batch"], c["hq"], c["dim"], dtype=torch.float64, device=DEV)
        lse = torch.full((c["batch"], c["hq"]), INF, dtype=torch.float64, device=DEV)
        w = s["w_out"].double()
        for b, n in enumerate(lens):
            if n == 0:
                continue
            at = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
            rows = s["table"][b, :-(-n // page)].long()
            k, v = (t[rows].flatten(0, 1)[at:n].double().repeat_interleave(g, 1) for t in (s["kc"], s["vc"]))
            x = (k * s["q"][b].double()).sum(-1).T / math.sqrt(c["dim"])  # [hq, keys]
            x = c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] > 0 else x
            lse[b] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b][:, None])
            out[b] = (p.T.unsqueeze(-1) * v).sum(0)
            w[b, :, :n] = s["w"][b, :, :n].double()
            w[b, :, at:n] += p.view(c["hk"], g, -1).sum(1)
        return {"out": out, "lse": lse, "weights": w} if c["weights"] else {"out": out, "lse": lse}
    w, slots, out = s["w_out"].double(), s["slots_out"], s["seqlens"].clone()
    kc, vc = s["kc"].double(), s["vc"].double()
    for b, n in enumerate(lens):
        m = min(n, c["budget"])
        out[b] = m
        rows = s["table"][b].long()
        for h in range(c["hk"]):
            rank = s["w"][b, h, :n].double()
            rank[s["slots"][b, h, :n] >= n - c["recent"]] = INF  # `seen` is the length here
            keep = (-rank).argsort(stable=True)[:m].sort().values
            low, moved = keep[keep < m], keep[keep >= m]
            at = torch.arange(m, device=DEV)
            free = at[~torch.isin(at, low)]
            w[b, h, :n], slots[b, h, :n] = 0.0, -1
            w[b, h, low], w[b, h, free] = s["w"][b, h, low].double(), s["w"][b, h, moved].double()
            slots[b, h, low], slots[b, h, free] = s["slots"][b, h, low], s["slots"][b, h, moved]
            for t in (kc, vc):
                t[rows[free // page], free % page, h] = t[rows[moved // page], moved % page, h]
    return {"k_cache": kc, "v_cache": vc, "seqlens": out, "weights": w, "slots": slots}
