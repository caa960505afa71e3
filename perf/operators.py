"""Cases of the paged key / value cache operators: rotary positions, appending to the cache, attention of new
tokens over it, and forking, growing and compacting its pages. ``run`` computes a case with elementary torch
operations, or (``own``) with the calls of ``attention_fa_fwd_02_gb300.kv``.

The cache of every case: K and V as [planes, pages, page, kv heads, D] (planes: the layers that share one page
table), a table [slots, pages of a slot] of page numbers (-1: none), a length per slot, a reference count per page.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
PHI = 0.6180339887498949


def listed():
    return [
        # q and k of a training step: 2 sequences of 4096 tokens, 32 / 8 heads of 128
        rope("rope-train", "bf16", 8192, 32, 8, 128, 128, "half", "none", 4096, False),
        # the gradient of a partial, interleaved rotation, fp32, odd number of far tokens
        rope("rope-grad-partial", "f32", 1537, 8, 8, 64, 32, "interleaved", "bands", 131072, True),
        # one decoding step of 48 sequences: the new token of each rotated and written
        append("append-decode", "bf16", 48, 1, 0, 16384, 32, 8, 128, 16, "half", "yarn"),
        # ragged chunks of up to 1024 new tokens for 8 sequences
        append("append-chunks", "bf16", 8, 1024, 7, 16384, 16, 4, 128, 32, "interleaved", "none"),
        # a single user's decoding step over a short context: latency
        attend("attend-single", "bf16", 1, 1, 0, 1021, 16, 4, 128, 16, 0),
        # a served batch: 64 sequences of up to 16384 tokens, one new token each
        attend("attend-batch", "bf16", 64, 1, 0, 16384, 32, 8, 128, 16, 0),
        # up to 5 drafted tokens to verify per sequence, fp32 cache, windowed, padded batch
        attend("attend-draft-f32", "f32", 12, 5, 9, 8000, 8, 8, 64, 32, 1024),
        # a long prompt's chunk: 2048 new tokens over 16384
        attend("attend-chunk", "bf16", 1, 2048, 0, 16384, 32, 8, 128, 64, 0),
        # four samples of one short prompt, each given its next token
        fork("fork-samples", "bf16", 1, 4, 1, 333, 1, 4, 128, 16),
        # beams of 32 sequences over 4 layers, each given 3 tokens
        fork("fork-beams", "bf16", 32, 4, 3, 2048, 4, 8, 128, 16),
        # a small cache closed up after sequences left
        compact("compact-small", "f32", 96, 40, 0.5, 1, 8, 64, 16),
        # 8192 pages of 2 layers, a third of the sequences gone
        compact("compact-large", "bf16", 8192, 128, 0.35, 2, 8, 128, 16),
    ]


def rope(name, dtype, T, H, HKV, D, rot, layout, scaling, far, grad):
    return dict(name=name, op="rope", dtype=dtype, T=T, H=H, HKV=HKV, D=D, rot=rot, layout=layout, scaling=scaling,
                far=far, grad=grad)


def append(name, dtype, B, n, pad, L, H, HKV, D, page, layout, scaling):
    return dict(name=name, op="append", dtype=dtype, B=B, n=n, pad=pad, L=L, H=H, HKV=HKV, D=D, page=page,
                layout=layout, scaling=scaling)


def attend(name, dtype, B, n, pad, L, H, HKV, D, page, window):
    return dict(name=name, op="attend", dtype=dtype, B=B, n=n, pad=pad, L=L, H=H, HKV=HKV, D=D, page=page,
                window=window)


def fork(name, dtype, B, ways, add, L, planes, HKV, D, page):
    return dict(name=name, op="fork", dtype=dtype, B=B, ways=ways, add=add, L=L, planes=planes, HKV=HKV, D=D,
                page=page)


def compact(name, dtype, pages, B, gone, planes, HKV, D, page):
    return dict(name=name, op="compact", dtype=dtype, pages=pages, B=B, gone=gone, planes=planes, HKV=HKV, D=D,
                page=page)


def draw(rng):
    def logint(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([32, 64, 80, 96, 128, 128])
    HKV = rng.choice([1, 2, 4, 5, 8])
    H = HKV * rng.choice([1, 2, 3, 4, 8] if HKV < 8 else [1, 2, 4])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    layout, scaling = rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "ntk", "bands", "yarn"])
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "fork", "compact"])
    if op == "rope":
        c = rope("", dtype, logint(1, 8000), H, HKV, D, rng.choice([D, D // 2, D // 4 * 2]), layout, scaling,
                 logint(4096, 1 << 20), rng.random() < 0.5)
    elif op == "append":
        B = logint(1, 64)
        c = append("", dtype, B, logint(1, max(2, 4096 // B)), rng.randrange(9), logint(5000, 16384), H, HKV, D, page,
                   layout, scaling)
    elif op == "attend":
        B = logint(1, 64)
        n = 1 if rng.random() < 0.4 else logint(2, max(3, 2048 // B))
        if dtype == "f32":
            n = min(n, 8)
        c = attend("", dtype, B, n, rng.randrange(9), max(n, logint(100, 16384 if B * n < 512 and dtype == "bf16" else 8192)),
                   H, HKV, D, page, rng.choice([0, 0, 0, logint(16, 4096)]))
    elif op == "fork":
        c = fork("", dtype, logint(1, 32), rng.randrange(2, 5), logint(1, 40), logint(20, 2000), rng.randrange(1, 5),
                 min(HKV, 8), D, min(page, 64))
    else:
        B = logint(4, 128)
        c = compact("", dtype, B * logint(4, 40), B, rng.choice([0.2, 0.35, 0.5, 0.8]), rng.randrange(1, 3), HKV, D,
                    min(page, 32))
    del c["name"]
    return c


def lengths(B, top, least=1):
    """B lengths from `least` to `top`, spread evenly; the first is `top`."""
    return [max(least, int(round(top * (1.0 - (b * PHI) % 1.0)))) for b in range(B)]


def sizes(c):
    """New tokens and lengths (new ones included) of the sequences of an append or attend case."""
    new = lengths(c["B"], c["n"])
    return new, [max(a, b) for a, b in zip(new, lengths(c["B"], c["L"]))]


def scaling_of(c):
    return {"none": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=8.0),
            "bands": dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192),
            "yarn": dict(kind="yarn", factor=16.0, beta_fast=32.0, beta_slow=1.0, original=4096)}[c["scaling"]]


def base_of(c):
    return 500000.0 if c["scaling"] == "bands" else 10000.0


def angles(rot, base, s, device):
    """Frequencies of the rot / 2 pairs in radians a token, in 64 bits, and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    kind = s["kind"] if s else "none"
    if kind == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if kind == "linear":
        return f / s["factor"], 1.0
    if kind == "bands":  # short waves as they are, long ones slowed, the band between in proportion
        turns = s["original"] * f / (2 * math.pi)
        t = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0.0, 1.0)
        return f * ((1 - t) / s["factor"] + t), 1.0
    if kind == "yarn":  # the ramp runs over pair numbers
        lo = math.floor(rot * math.log(s["original"] / (2 * math.pi * s["beta_fast"])) / (2 * math.log(base)))
        hi = math.ceil(rot * math.log(s["original"] / (2 * math.pi * s["beta_slow"])) / (2 * math.log(base)))
        lo, hi = max(lo, 0), min(hi, rot - 1)
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (t / s["factor"] + 1 - t), 0.1 * math.log(s["factor"]) + 1.0
    return f, 1.0


def paged(c, slots, width, lens, planes, extra, g, fill):
    """A cache whose first slots have `lens` tokens, their pages in an order of the seed's, `extra` pages free."""
    dev, page = "cuda", c["page"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    at = torch.arange(width, device=dev)
    first = torch.tensor([0] + need, device=dev).cumsum(0)
    table = torch.full((slots, width), -1, dtype=torch.int32, device=dev)
    used = at < torch.tensor(need, device=dev)[:, None]
    table[:len(lens)][used] = order[(first[:-1, None] + at)[used]]
    length = torch.zeros(slots, dtype=torch.int32, device=dev)
    length[:len(lens)] = torch.tensor(lens, dtype=torch.int32, device=dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[order[:sum(need)].long()] = 1
    shape = (planes, pages, page, c["HKV"], c["D"])
    k = torch.randn(shape, generator=g, device=dev, dtype=DT[c["dtype"]]) * fill
    v = torch.randn(shape, generator=g, device=dev, dtype=DT[c["dtype"]])
    return dict(k=k, v=v, table=table, lens=length, refs=refs)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * mul).to(dt)

    if c["op"] == "rope":
        s = dict(q=normal(c["T"], c["H"], c["D"]), k=normal(c["T"], c["HKV"], c["D"]),
                 pos=torch.randint(0, c["far"], (c["T"],), generator=g, device="cuda"))
    elif c["op"] in ("append", "attend"):
        new, lens = sizes(c)
        width = -(-max(lens) // c["page"]) + 1
        s = paged(c, c["B"], width, lens, 1, 3, g, 1.5 if c["op"] == "attend" else 1.0)
        T = sum(new) + c["pad"]
        s.update(q=normal(T, c["H"], c["D"], mul=1.5 if c["op"] == "attend" else 1.0), T=sum(new),
                 cu=torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32),
                 o=torch.zeros(T, c["H"], c["D"], dtype=dt, device="cuda"))
        if c["op"] == "append":
            s.update(kn=normal(T, c["HKV"], c["D"]), vn=normal(T, c["HKV"], c["D"]))
        else:
            s.update(lse=torch.zeros(T, c["H"], device="cuda"))
    elif c["op"] == "fork":
        lens = lengths(c["B"], c["L"])
        slots = c["B"] * c["ways"]
        width = -(-(max(lens) + c["add"]) // c["page"]) + 1
        s = paged(c, slots, width, lens, c["planes"], slots * (c["add"] // c["page"] + 2), g, 1.0)
        # the first sample goes on in its own slot, the others are forked from it
        src = torch.arange(c["B"], device="cuda").repeat_interleave(c["ways"] - 1)
        s.update(src=src.to(torch.int32),
                 dst=torch.arange(c["B"], slots, device="cuda", dtype=torch.int32),
                 add=torch.full((slots - c["B"],), c["add"], dtype=torch.int32, device="cuda"))
    else:
        per = lengths(c["B"], 2 * c["pages"] // c["B"] - 1)
        lens = [n * c["page"] - (b % c["page"]) for b, n in enumerate(per)]
        s = paged(c, c["B"], max(per) + 1, lens, c["planes"], 5, g, 1.0)
        gone = torch.rand(c["B"], generator=g, device="cuda") < c["gone"]
        left = s["table"][gone]
        s["refs"][left[left >= 0].long()] = 0
        s["table"][gone] = -1
        s["lens"][gone] = 0
        s.update(table0=s["table"].clone(), refs0=s["refs"].clone())
    s["case"] = c
    if own:
        from attention_fa_fwd_02_gb300 import kv
        if c["op"] != "rope":
            s["cache"] = kv.PagedCache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
        if "scaling" in c:
            s["rope"] = kv.Rope(c["D"], c.get("rot", c["D"]), base_of(c), c["layout"], scaling_of(c))
    elif "scaling" in c:
        s["freqs"], s["mscale"] = angles(c.get("rot", c["D"]), base_of(c), scaling_of(c), "cuda")
    return s


def run(s):
    c = s["case"]
    if own:
        if c["op"] == "rope":
            return s["rope"].apply(s["q"], s["k"], s["pos"], inverse=c["grad"])
        cache = s["cache"]
        if c["op"] == "append":
            q = cache.append(s["q"], s["kn"], s["vn"], s["cu"], rope=s["rope"], out=s["o"])
            return q, s["k"], s["v"]
        if c["op"] == "attend":
            return cache.attend(s["q"], s["cu"], window=c["window"], out=s["o"], lse=s["lse"])
        if c["op"] == "fork":
            cache.fork(s["src"], s["dst"])
            cache.grow(s["dst"], s["add"])
        else:
            s["table"].copy_(s["table0"])  # the state before sequences left is the same for each pass
            s["refs"].copy_(s["refs0"])
            cache.compact()
    elif c["op"] == "rope":
        return tuple(rotated(x, s["pos"], s, c["rot"], -1.0 if c["grad"] else 1.0) for x in (s["q"], s["k"]))
    elif c["op"] == "append":
        seq, pos = tokens(s, c)
        n, page = s["T"], s["table"][seq, pos // c["page"]].long()
        s["o"][:n] = rotated(s["q"][:n], pos, s, c["D"], 1.0)
        s["k"][0, page, pos % c["page"]] = rotated(s["kn"][:n], pos, s, c["D"], 1.0)
        s["v"][0, page, pos % c["page"]] = s["vn"][:n]
        return s["o"], s["k"], s["v"]
    elif c["op"] == "attend":
        return attended(s, c)
    elif c["op"] == "fork":
        forked(s, c)
        grown(s, c)
    else:
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        compacted(s)
    return {x: s[x] for x in ("table", "lens", "refs", "k", "v")}


# ---- the plain forms


def rotated(x, pos, s, rot, sign):
    """x [T, heads, D] with its first `rot` columns turned by sign * pos * frequency."""
    a = pos.double()[:, None, None] * s["freqs"]
    cos, sin = (a.cos() * s["mscale"]).float(), (a.sin() * (sign * s["mscale"])).float()
    y = x.float()
    if s["case"]["layout"] == "half":
        u, w = y[..., :rot // 2], y[..., rot // 2:rot]
        y = torch.cat([u * cos - w * sin, w * cos + u * sin, y[..., rot:]], -1)
    else:
        u, w = y[..., 0:rot:2], y[..., 1:rot:2]
        y = torch.cat([torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2), y[..., rot:]], -1)
    return y.to(x.dtype)


def tokens(s, c):
    """Sequence and position of every new token."""
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), new, output_size=s["T"])
    at = torch.arange(s["T"], device="cuda") - s["cu"].long()[seq]
    return seq, s["lens"].long()[seq] - new[seq] + at


def attended(s, c):
    seq, pos = tokens(s, c)
    B, H, HKV, D, n = c["B"], c["H"], c["HKV"], c["D"], max(lengths(c["B"], c["n"]))
    at = torch.arange(s["T"], device="cuda") - s["cu"].long()[seq]
    q = torch.zeros(B, n, H, D, device="cuda")
    q[seq, at] = s["q"][:s["T"]].float()
    p = torch.full((B, n), -1, dtype=torch.long, device="cuda")
    p[seq, at] = pos
    rows = s["table"].long().clamp(min=0)
    j = torch.arange(rows.shape[1] * c["page"], device="cuda")
    k, v = (x[0][rows].float().reshape(B, -1, HKV, D) for x in (s["k"], s["v"]))
    q = q.reshape(B, n, HKV, H // HKV, D).permute(0, 2, 3, 1, 4).reshape(B, HKV, -1, D)
    z = q @ k.permute(0, 2, 3, 1) * (1.0 / math.sqrt(D))
    see = j <= p[..., None]
    if c["window"]:
        see &= j > p[..., None] - c["window"]
    z = z.reshape(B, HKV, H // HKV, n, -1).masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    w = z.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.reshape(B, HKV, -1, w.shape[-1]) @ v.permute(0, 2, 1, 3)).reshape(B, HKV, H // HKV, n, D)
    o = (o / total).permute(0, 3, 1, 2, 4).reshape(B, n, H, D)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, n, H)
    s["o"][:s["T"]] = o[seq, at].to(s["o"].dtype)
    s["lse"][:s["T"]] = lse[seq, at]
    return s["o"], s["lse"]


def forked(s, c):
    """The slots dst become copies of the slots src, which share their pages."""
    src, dst, table, refs = s["src"].long(), s["dst"].long(), s["table"], s["refs"]
    rows, old = table[src], table[dst]
    one = torch.ones((), dtype=torch.int32, device="cuda")
    held = rows[rows >= 0].long()
    refs.index_add_(0, held, one.expand(held.shape[0]))
    left = old[old >= 0].long()
    refs.index_add_(0, left, -one.expand(left.shape[0]))
    table[dst] = rows
    s["lens"][dst] = s["lens"][src]


def grown(s, c):
    """Room for `add` more tokens in the slots dst: the lowest free pages, a shared last page replaced by a copy."""
    slots, add, table, refs, page = s["dst"].long(), s["add"].long(), s["table"], s["refs"], c["page"]
    have = s["lens"].long()[slots]
    old, new = (have + page - 1) // page, (have + add + page - 1) // page
    tail = table[slots, (have // page).clamp(max=table.shape[1] - 1)].long().clamp(min=0)
    copy = (have % page != 0) & (add > 0) & (refs[tail] > 1)
    need = new - old + copy
    first = need.cumsum(0) - need
    free = torch.nonzero(refs == 0)[:, 0]
    i = torch.repeat_interleave(torch.arange(slots.shape[0], device="cuda"), need)
    at = torch.arange(i.shape[0], device="cuda")
    got = free[:i.shape[0]]
    fresh = got[first[copy]]
    s["k"][:, fresh] = s["k"][:, tail[copy]]
    s["v"][:, fresh] = s["v"][:, tail[copy]]
    refs.index_add_(0, tail[copy], -torch.ones_like(fresh, dtype=torch.int32))
    refs[got] = 1
    table[slots[i], old[i] + at - first[i] - copy[i].long()] = got.to(torch.int32)
    s["lens"][slots] += s["add"]


def compacted(s):
    """Live pages beyond the number of live pages go to the free ones below it, in order."""
    live = s["refs"] > 0
    n = live.sum()
    at = torch.arange(live.shape[0], device="cuda")
    src, dst = torch.nonzero(live & (at >= n))[:, 0], torch.nonzero(~live & (at < n))[:, 0]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["refs"][dst] = s["refs"][src]
    s["refs"][src] = 0
    t = s["table"]
    t.copy_(torch.where(t >= 0, to[t.long().clamp(min=0)], t))


# ---- from the definitions, in 64 bits


def exact(case, seed):
    c = dict(case)
    if c["op"] == "rope":
        s = without_own(case, seed)
        turn = exact_angles(s["pos"].double(), c, c["rot"], -1.0 if c["grad"] else 1.0)
        return tuple(exact_turn(s[x].double(), turn, c["layout"]) for x in ("q", "k"))
    if c["op"] == "append":
        s = without_own(case, seed)
        new, lens = sizes(c)
        q, k, v = s["o"].double(), s["k"].double(), s["v"].double()
        at = 0
        for b in range(c["B"]):
            p = torch.arange(lens[b] - new[b], lens[b], device="cuda")
            turn = exact_angles(p.double(), c, c["D"], 1.0)
            t = slice(at, at + new[b])
            q[t] = exact_turn(s["q"][t].double(), turn, c["layout"])
            where = s["table"][b].long()[torch.div(p, c["page"], rounding_mode="floor")]
            k[0, where, p % c["page"]] = exact_turn(s["kn"][t].double(), turn, c["layout"])
            v[0, where, p % c["page"]] = s["vn"][t].double()
            at += new[b]
        return q, k, v
    if c["op"] == "attend":
        if work(case)["flops"] > 1.2e12:
            return None
        s = without_own(case, seed)
        new, lens = sizes(c)
        o, lse = s["o"].double(), s["lse"].double()
        group, at = c["H"] // c["HKV"], 0
        for b in range(c["B"]):
            rows = s["table"][b, :-(-lens[b] // c["page"])].long()
            k, v = (s[x][0][rows].reshape(-1, c["HKV"], c["D"])[:lens[b]] for x in ("k", "v"))
            for h in range(c["HKV"]):
                kh, vh = k[:, h].double(), v[:, h].double()
                for a in range(0, new[b], 512):
                    e = min(a + 512, new[b])
                    q = s["q"][at + a:at + e, h * group:(h + 1) * group].double()
                    p = torch.arange(lens[b] - new[b] + a, lens[b] - new[b] + e, device="cuda")
                    gap = p[:, None, None] - torch.arange(lens[b], device="cuda")
                    hide = gap < 0
                    if c["window"]:
                        hide = hide | (gap >= c["window"])
                    z = torch.einsum("tgd,jd->tgj", q, kh) / math.sqrt(c["D"])
                    z = z.masked_fill(hide, -math.inf)
                    lse[at + a:at + e, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
                    o[at + a:at + e, h * group:(h + 1) * group] = torch.softmax(z, -1) @ vh
            at += new[b]
        return o, lse
    return None  # whole numbers and copies: nothing is computed


def without_own(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def exact_angles(pos, c, rot, sign):
    """cos, sin [T, rot / 2] of the scaled rotation, each pair's frequency by itself."""
    f, s, base = [], scaling_of(c), base_of(c)
    for i in range(rot // 2):
        x = math.pow(base, -2.0 * i / rot)
        if s and s["kind"] == "linear":
            x /= s["factor"]
        elif s and s["kind"] == "ntk":
            x = math.pow(base * math.pow(s["factor"], rot / (rot - 2.0)), -2.0 * i / rot)
        elif s and s["kind"] == "bands":
            wave = 2 * math.pi / x
            if wave > s["original"] / s["low"]:
                x /= s["factor"]
            elif wave > s["original"] / s["high"]:
                part = (s["original"] / wave - s["low"]) / (s["high"] - s["low"])
                x = (1 - part) * x / s["factor"] + part * x
        elif s and s["kind"] == "yarn":
            edge = [rot * math.log(s["original"] / (b * 2 * math.pi)) / (2 * math.log(base))
                    for b in (s["beta_fast"], s["beta_slow"])]
            low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            part = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            x = x / s["factor"] * part + x * (1 - part)
        f.append(x)
    a = pos[:, None] * torch.tensor(f, dtype=torch.float64, device=pos.device)
    m = 0.1 * math.log(s["factor"]) + 1.0 if s and s["kind"] == "yarn" else 1.0
    return m * torch.cos(a), m * sign * torch.sin(a)


def exact_turn(x, turn, layout):
    cos, sin = (t[:, None] for t in turn)
    half = cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y[..., a] = cos * x[..., a] - sin * x[..., b]
    y[..., b] = sin * x[..., a] + cos * x[..., b]
    return y


# ---- what a pass cannot do without


def work(case):
    c, e = case, ES[case["dtype"]]
    token = c["HKV"] * c["D"] * e  # bytes of K (or V) of a token in one plane
    if c["op"] == "rope":
        x = c["T"] * (c["H"] + c["HKV"]) * c["D"]
        return {"bytes": 2 * x * e + 8 * c["T"], "flops": 3 * x}
    if c["op"] == "append":
        T = sum(sizes(c)[0])
        return {"bytes": 2 * T * (c["H"] * c["D"] * e + 2 * token), "flops": 3 * T * (c["H"] + c["HKV"]) * c["D"]}
    if c["op"] == "attend":
        new, lens = sizes(c)
        w = c["window"] or 1 << 40
        keys = sum(min(n, w + a - 1) for a, n in zip(new, lens))
        pairs = sum(seen(n, w) - seen(n - a, w) for a, n in zip(new, lens))
        T = sum(new)
        return {"bytes": 2 * keys * token + T * c["H"] * (2 * c["D"] * e + 4) + 4 * keys // c["page"],
                "flops": 4 * c["H"] * c["D"] * pairs}
    pagebytes = 2 * c["planes"] * c["page"] * token
    if c["op"] == "fork":
        lens = lengths(c["B"], c["L"])
        copies = sum(n % c["page"] != 0 for n in lens) * (c["ways"] - 1)
        rows = sum(-(-n // c["page"]) for n in lens) * (1 + c["ways"] - 1)
        return {"bytes": 2 * copies * pagebytes + 12 * rows, "flops": 0}
    used = sum(lengths(c["B"], 2 * c["pages"] // c["B"] - 1))
    live = int(used * (1 - c["gone"]))
    moved = live * (used + 5 - live) // (used + 5)
    return {"bytes": 2 * moved * pagebytes + 12 * used, "flops": 0}


def seen(n, w):
    """Visible pairs of positions 0 .. n - 1 under a window of w."""
    m = min(n, w)
    return m * (m + 1) // 2 + (n - m) * m


if __name__ == "__main__":  # the cases and their floors' bytes and operations
    for case in listed() + [draw(random.Random(x)) for x in range(6)]:
        print(case, work(case))
