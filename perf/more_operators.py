"""Cases of a paged key / value cache held in 4 or 8 bits: new tokens quantised as they are written, the cache read
back, and attention of new tokens over it. ``run`` computes a case with elementary torch operations, or (``own``) with
the calls of ``attention_fa_fwd_02_gb300.kv``.

What a cache holds of a token's K or V row x [D] of one head: for each group of G columns a scale s and an offset z,
both bf16, and a code c in 0 .. L = 2^bits - 1 per column, which stands for s c + z:
    z = the largest bf16 <= min x,  s = the smallest bf16 >= (max x - z) / L,  c = round((x - z) / s), ties to even
(s = 0: c = 0). The table [slots, pages of a slot] has page numbers (-1: none); there is a length per slot.
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
        # one decoding step of 48 sequences: the new token of each rotated, quantised, written and read back
        append("qappend-decode", "bf16", 48, 1, 0, 16384, 32, 8, 128, 16, 4, 64, "half", "yarn"),
        # ragged chunks of up to 1024 new tokens for 8 sequences, in 8 bits
        append("qappend-chunks", "bf16", 8, 1024, 7, 16384, 16, 4, 128, 32, 8, 128, "interleaved", "none"),
        # the prefix of one sequence as contiguous K and V, for a pass over it that needs them
        read("qread-prefix", "bf16", 1, 1021, 4, 128, 16, 4, 64),
        # 8 sequences of up to 16384 tokens handed on in fp32, odd head dim
        read("qread-all-f32", "f32", 8, 16384, 5, 80, 64, 8, 80),
        # a single user's decoding step over a short context: latency
        attend("qattend-single", "bf16", 1, 1, 0, 1021, 16, 4, 128, 16, 4, 64, 0),
        # a served batch: 64 sequences of up to 16384 tokens in 4 bits, one new token each
        attend("qattend-batch4", "bf16", 64, 1, 0, 16384, 32, 8, 128, 16, 4, 64, 0),
        # 32 sequences of up to 8192 tokens in 8 bits
        attend("qattend-batch8", "bf16", 32, 1, 0, 8192, 32, 8, 128, 32, 8, 128, 0),
        # up to 5 drafted tokens to verify per sequence, fp32 queries, windowed, padded batch
        attend("qattend-draft-f32", "f32", 12, 5, 9, 8000, 8, 8, 64, 32, 8, 64, 1024),
        # up to 4 drafted tokens for 16 sequences of up to 8192
        attend("qattend-draft4", "bf16", 16, 4, 0, 8192, 32, 8, 128, 16, 4, 128, 0),
        # a long prompt's chunk: 2048 new tokens over 16384 in 4 bits
        attend("qattend-chunk4", "bf16", 1, 2048, 0, 16384, 32, 8, 128, 64, 4, 64, 0),
        # ragged chunks of up to 500 tokens for 6 sequences in 8 bits, odd head dim
        attend("qattend-chunks8", "bf16", 6, 500, 3, 5000, 12, 4, 96, 32, 8, 96, 0),
    ]


def append(name, dtype, B, n, pad, L, H, HKV, D, page, bits, group, layout, scaling):
    return dict(name=name, op="append", dtype=dtype, B=B, n=n, pad=pad, L=L, H=H, HKV=HKV, D=D, page=page, bits=bits,
                group=group, layout=layout, scaling=scaling)


def read(name, dtype, B, L, HKV, D, page, bits, group):
    return dict(name=name, op="read", dtype=dtype, B=B, n=L, pad=0, L=L, H=HKV, HKV=HKV, D=D, page=page, bits=bits,
                group=group)


def attend(name, dtype, B, n, pad, L, H, HKV, D, page, bits, group, window):
    return dict(name=name, op="attend", dtype=dtype, B=B, n=n, pad=pad, L=L, H=H, HKV=HKV, D=D, page=page, bits=bits,
                group=group, window=window)


def draw(rng):
    def logint(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    dtype, bits = rng.choice(["bf16", "bf16", "f32"]), rng.choice([4, 4, 8])
    D = rng.choice([32, 64, 80, 96, 128, 128])
    group = 64 if D == 128 and rng.random() < 0.5 else D
    HKV = rng.choice([1, 2, 4, 5, 8])
    H = HKV * rng.choice([1, 2, 3, 4, 8] if HKV < 8 else [1, 2, 4])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    B = logint(1, 64)
    if op == "append":
        c = append("", dtype, B, logint(1, max(2, 4096 // B)), rng.randrange(9), logint(5000, 16384), H, HKV, D, page,
                   bits, group, rng.choice(["half", "interleaved"]),
                   rng.choice(["none", "linear", "ntk", "bands", "yarn"]))
    elif op == "read":
        c = read("", dtype, min(B, 16), logint(20, 8192), HKV, D, page, bits, group)
    else:
        n = 1 if rng.random() < 0.4 else logint(2, max(3, 2048 // B))
        if dtype == "f32":
            n = min(n, 8)
        c = attend("", dtype, B, n, rng.randrange(9),
                   max(n, logint(100, 16384 if B * n < 512 and dtype == "bf16" else 8192)), H, HKV, D, page, bits,
                   group, rng.choice([0, 0, 0, logint(16, 4096)]))
    del c["name"]
    return c


def lengths(B, top, least=1):
    """B lengths from `least` to `top`, spread evenly; the first is `top`."""
    return [max(least, int(round(top * (1.0 - (b * PHI) % 1.0)))) for b in range(B)]


def sizes(c):
    """New tokens (read: all of them) and lengths, new ones included, of the sequences of a case."""
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
    if kind == "bands":
        turns = s["original"] * f / (2 * math.pi)
        t = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0.0, 1.0)
        return f * ((1 - t) / s["factor"] + t), 1.0
    if kind == "yarn":
        lo = math.floor(rot * math.log(s["original"] / (2 * math.pi * s["beta_fast"])) / (2 * math.log(base)))
        hi = math.ceil(rot * math.log(s["original"] / (2 * math.pi * s["beta_slow"])) / (2 * math.log(base)))
        lo, hi = max(lo, 0), min(hi, rot - 1)
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (t / s["factor"] + 1 - t), 0.1 * math.log(s["factor"]) + 1.0
    return f, 1.0


def prepare(case, seed):
    c = dict(case)
    dev, dt, page = "cuda", DT[c["dtype"]], c["page"]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, mul=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt).mul_(mul)

    def cu_of(counts):
        return torch.tensor([0] + counts, device=dev).cumsum(0).to(torch.int32)

    new, lens = sizes(c)
    if c["op"] == "read":
        new = lens
    # pages in an order of the seed's, three of them free
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    at = torch.arange(width, device=dev)
    first = torch.tensor([0] + need, device=dev).cumsum(0)
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=dev)
    used = at < torch.tensor(need, device=dev)[:, None]
    table[used] = order[(first[:-1, None] + at)[used]]
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[order[:sum(need)].long()] = 1
    s = dict(case=c, T=sum(new), cu=cu_of(new), table=table, refs=refs,
             lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    rows = s["T"] + c["pad"]
    if c["op"] == "append":
        s.update(q=normal(rows, c["H"], c["D"]), kn=normal(rows, c["HKV"], c["D"]), vn=normal(rows, c["HKV"], c["D"]),
                 o=torch.zeros(rows, c["H"], c["D"], dtype=dt, device=dev),
                 back=[torch.zeros(s["T"], c["HKV"], c["D"], dtype=torch.bfloat16, device=dev) for _ in range(2)])
    elif c["op"] == "read":
        s.update(back=[torch.zeros(s["T"], c["HKV"], c["D"], dtype=dt, device=dev) for _ in range(2)])
    else:
        s.update(q=normal(rows, c["H"], c["D"], mul=1.5), o=torch.zeros(rows, c["H"], c["D"], dtype=dt, device=dev),
                 lse=torch.zeros(rows, c["H"], device=dev))
    k = v = None
    if c["op"] != "append":  # what the cache holds already
        k, v = normal(sum(lens), c["HKV"], c["D"], mul=1.5), normal(sum(lens), c["HKV"], c["D"])
    if own:
        from attention_fa_fwd_02_gb300 import kv
        s["cache"] = kv.QuantCache.create(1, pages, page, c["HKV"], c["D"], c["B"], width, bits=c["bits"],
                                          group=c["group"], dtype=dt)
        for x in ("table", "lens", "refs"):
            getattr(s["cache"], x).copy_(s[x])
        if k is not None:
            s["cache"].append(None, k, v, cu_of(lens))
        else:
            s["rope"] = kv.Rope(c["D"], c["D"], base_of(c), c["layout"], scaling_of(c))
    else:
        shape = (pages, page, c["HKV"])
        for x in "kv":
            s[x] = (torch.zeros(*shape, c["D"] * c["bits"] // 8, dtype=torch.uint8, device=dev),
                    torch.zeros(*shape, c["D"] // c["group"], 2, dtype=torch.bfloat16, device=dev))
        if k is not None:
            seq = torch.repeat_interleave(torch.arange(c["B"], device=dev), s["lens"].long())
            pos = torch.arange(sum(lens), device=dev) - cu_of(lens)[:-1].long()[seq]
            put(s, seq, pos, k, v)
        else:
            s["freqs"], s["mscale"] = angles(c["D"], base_of(c), scaling_of(c), dev)
    return s


def run(s):
    c = s["case"]
    if own:
        cache = s["cache"]
        if c["op"] == "append":
            q = cache.append(s["q"], s["kn"], s["vn"], s["cu"], rope=s["rope"], out=s["o"])
            return q, *cache.read(s["cu"], s["T"], out=s["back"])
        if c["op"] == "read":
            return cache.read(s["cu"], s["T"], out=s["back"])
        return cache.attend(s["q"], s["cu"], window=c["window"], out=s["o"], lse=s["lse"])
    if c["op"] == "attend":
        return attended(s, c)
    seq, pos = tokens(s, c)
    if c["op"] == "append":
        n = s["T"]
        s["o"][:n] = rotated(s["q"][:n], pos, s).to(s["o"].dtype)
        put(s, seq, pos, rotated(s["kn"][:n], pos, s), s["vn"][:n])
    page, row = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    for x, to in zip("kv", s["back"]):
        codes, params = s[x]
        to.copy_(values(codes[page, row], params[page, row], c))
    return (s["o"], *s["back"]) if c["op"] == "append" else s["back"]


# ---- the plain forms


def down(x):
    """The largest bf16 values <= x, as fp32."""
    i = x.contiguous().view(torch.int32)
    cut = i & -65536
    return torch.where((i != cut) & (i < 0), cut + 65536, cut).view(torch.float32)


def quantised(x, c):
    """Codes packed into bytes (4 bits: even columns low) and (scale, offset) of x [..., D]."""
    x = x.float().unflatten(-1, (-1, c["group"]))
    top = 2 ** c["bits"] - 1
    z = down(x.amin(-1))
    s = -down((z - x.amax(-1)) / torch.full_like(z, top))  # (a quotient: a number would be turned into its reciprocal)
    code = torch.where(s[..., None] > 0, ((x - z[..., None]) / s[..., None]).round_().clamp_(0, top), 0.0)
    code = code.flatten(-2).to(torch.uint8)
    if c["bits"] == 4:
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code, torch.stack([s, z], -1).to(torch.bfloat16)


def values(codes, params, c):
    if c["bits"] == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    p = params.float()
    return (codes.float().unflatten(-1, (-1, c["group"])) * p[..., :1] + p[..., 1:]).flatten(-2)


def put(s, seq, pos, k, v):
    page, row = s["table"][seq, pos // s["case"]["page"]].long(), pos % s["case"]["page"]
    for x, new in (("k", k), ("v", v)):
        codes, params = quantised(new, s["case"])
        s[x][0][page, row] = codes
        s[x][1][page, row] = params


def rotated(x, pos, s):
    """x [T, heads, D] turned by its positions, in fp32."""
    a = pos.double()[:, None, None] * s["freqs"]
    cos, sin = (a.cos() * s["mscale"]).float(), (a.sin() * s["mscale"]).float()
    y = x.float()
    if s["case"]["layout"] == "half":
        u, w = y.chunk(2, -1)
        return torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    u, w = y[..., 0::2], y[..., 1::2]
    return torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)


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
    k, v = (values(codes[rows], params[rows], c).reshape(B, -1, HKV, D) for codes, params in (s["k"], s["v"]))
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


# ---- from the definitions, in 64 bits


def exact(case, seed):
    c = dict(case)
    if c["op"] == "attend" and work(case)["flops"] > 1.2e12:
        return None
    s = without_own(case, seed)
    new, lens = sizes(c)
    if c["op"] == "append":
        q, k, v, at = s["o"].double(), [], [], 0
        for b in range(c["B"]):
            p = torch.arange(lens[b] - new[b], lens[b], dtype=torch.float64, device="cuda")
            turn = exact_angles(p, c)
            t = slice(at, at + new[b])
            q[t] = exact_turn(s["q"][t].double(), turn, c["layout"])
            k.append(exact_held(exact_turn(s["kn"][t].double(), turn, c["layout"]), c))
            v.append(exact_held(s["vn"][t].double(), c))
            at += new[b]
        return q, torch.cat(k), torch.cat(v)
    if c["op"] == "read":
        return [torch.cat([exact_rows(s, c, x, b, lens[b]) for b in range(c["B"])]) for x in "kv"]
    o, lse = s["o"].double(), s["lse"].double()
    rep, at = c["H"] // c["HKV"], 0
    for b in range(c["B"]):
        k, v = exact_rows(s, c, "k", b, lens[b]), exact_rows(s, c, "v", b, lens[b])
        for h in range(c["HKV"]):
            for a in range(0, new[b], 512):
                e = min(a + 512, new[b])
                q = s["q"][at + a:at + e, h * rep:(h + 1) * rep].double()
                p = torch.arange(lens[b] - new[b] + a, lens[b] - new[b] + e, device="cuda")
                gap = p[:, None, None] - torch.arange(lens[b], device="cuda")
                hide = gap < 0
                if c["window"]:
                    hide = hide | (gap >= c["window"])
                z = torch.einsum("tgd,jd->tgj", q, k[:, h]) / math.sqrt(c["D"])
                z = z.masked_fill(hide, -math.inf)
                lse[at + a:at + e, h * rep:(h + 1) * rep] = torch.logsumexp(z, -1)
                o[at + a:at + e, h * rep:(h + 1) * rep] = torch.softmax(z, -1) @ v[:, h]
        at += new[b]
    return o, lse


def without_own(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def exact_rows(s, c, x, b, n):
    """What the first n tokens of slot b hold, [n, HKV, D]."""
    at = torch.arange(n, device="cuda")
    page = s["table"][b].long()[torch.div(at, c["page"], rounding_mode="floor")]
    codes, params = (t[page, at % c["page"]] for t in s[x])
    col = torch.arange(c["D"], device="cuda")
    if c["bits"] == 4:
        code = torch.bitwise_right_shift(codes[..., col // 2].to(torch.int64), 4 * (col % 2)) % 16
    else:
        code = codes[..., col]
    p = params.double()[..., col // c["group"], :]
    return code.double() * p[..., 0] + p[..., 1]


def exact_held(x, c):
    """The values that stand for x [n, heads, D] in the cache."""
    y = torch.empty_like(x)
    steps = float(2 ** c["bits"] - 1)
    for g in range(0, c["D"], c["group"]):
        part = x[..., g:g + c["group"]]
        least, most = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        z = to_eight_bits(least, torch.floor)
        s = to_eight_bits((most - z) / steps, torch.ceil)
        code = torch.clamp(torch.round((part - z) / torch.where(s > 0, s, 1.0)), 0.0, steps)
        y[..., g:g + c["group"]] = s * code + z
    return y


def to_eight_bits(x, whole):
    """x to 8 significant bits, the last one rounded by `whole`."""
    m = torch.frexp(x).mantissa
    return torch.where(x == 0, x, whole(m * 256.0) * (x / m / 256.0))  # (x / m: the power of two, exact)


def exact_angles(pos, c):
    """cos, sin [T, D / 2] of the scaled rotation, each pair's frequency by itself."""
    rot, f, s, base = c["D"], [], scaling_of(c), base_of(c)
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
    return m * torch.cos(a), m * torch.sin(a)


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
    new, lens = sizes(c)
    values_ = c["HKV"] * c["D"]  # of K (or V) of a token
    held = c["HKV"] * (c["D"] * c["bits"] // 8 + 4 * c["D"] // c["group"])  # bytes of them in the cache
    T = sum(new)
    if c["op"] == "append":  # q in and out; K and V in, held, and out again in bf16
        return {"bytes": 2 * T * c["H"] * c["D"] * e + 2 * T * (values_ * (e + 2) + 2 * held),
                "flops": 3 * T * (c["H"] + c["HKV"]) * c["D"] + 8 * T * values_}
    if c["op"] == "read":
        T = sum(lens)
        return {"bytes": 2 * T * (held + values_ * e) + 4 * T // c["page"], "flops": 4 * T * values_}
    w = c["window"] or 1 << 40
    keys = sum(min(n, w + a - 1) for a, n in zip(new, lens))
    pairs = sum(seen(n, w) - seen(n - a, w) for a, n in zip(new, lens))
    return {"bytes": 2 * keys * held + T * c["H"] * (2 * c["D"] * e + 4) + 4 * keys // c["page"],
            "flops": 4 * c["H"] * c["D"] * pairs}


def seen(n, w):
    """Visible pairs of positions 0 .. n - 1 under a window of w."""
    m = min(n, w)
    return m * (m + 1) // 2 + (n - m) * m


if __name__ == "__main__":  # the cases and their floors' bytes and operations
    for case in listed() + [draw(random.Random(x)) for x in range(6)]:
        print(case, work(case))
