"""Plain references of the paged-cache operators: fp64 arithmetic and Python loops over sequences, tokens and
pages, with bounds on what the kernels' arithmetic may add."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def make_cache(kv, lens, page, HKV, D, dtype, seed=0, planes=1, slots=None, order=None, extra=3, layout="tokens",
               fill=1.5, max_pages=None, poison=True):
    """A cache whose slot order[b] (default b) holds lens[b] tokens on pages in a random order. Page memory that holds
    no token is NaN."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    slots = slots or B
    order = list(range(B)) if order is None else order
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    perm = torch.randperm(pages, generator=g).tolist()
    width = max_pages or max(need + [1]) + 1
    table = torch.full((slots, width), -1, dtype=torch.int32)
    length = torch.zeros(slots, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    shape = (planes, pages, page, HKV, D)
    k = torch.full(shape, float("nan") if poison else 0.0)
    v = torch.full(shape, float("nan") if poison else 0.0)
    at = 0
    for b, n in enumerate(lens):
        mine = perm[at:at + need[b]]
        at += need[b]
        table[order[b], :need[b]] = torch.tensor(mine, dtype=torch.int32)
        length[order[b]] = n
        for i, p in enumerate(mine):
            refs[p] = 1
            m = min(page, n - i * page)
            k[:, p, :m] = torch.randn(planes, m, HKV, D, generator=g) * fill
            v[:, p, :m] = torch.randn(planes, m, HKV, D, generator=g)
    if layout == "heads":
        k, v = k.transpose(2, 3).contiguous(), v.transpose(2, 3).contiguous()
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    return kv.PagedCache(k, v, table.cuda(), length.cuda(), refs.cuda(), layout)


def gather(cache, slot, plane=0, layout="tokens"):
    """K, V [len, HKV, D] fp64 of a slot."""
    n, page = int(cache.lens[slot]), cache.page_size
    rows = cache.table[slot, :-(-n // page)].long()
    out = []
    for x in (cache.k, cache.v):
        x = x[plane][rows]
        if layout == "heads":
            x = x.transpose(1, 2)
        out.append(x.reshape(-1, cache.kv_heads, cache.head_dim)[:n].double())
    return out


def attend(cache, q, new, slots, scale, causal, window, plane=0, layout="tokens", one_term=False):
    """O, LSE of the rows (fp64), and bounds on |O - ref| (before the output's rounding) and |LSE - ref|.

    Scores: products of the inputs are exact in fp32 (bf16) or good to 2^-21 (three tf32 products of rounded two-term
    splits: what is dropped is below 3 * 2^-23 of |q||k|), their sum of D terms errs by at most D 2^-23 of sum |q||k|
    (tensor-core sums need not round to nearest). A score error e moves its probability by the factor exp(e), so O_d by
    at most 2 e A_d, A_d = sum_j p_j |v_jd|, and the LSE by e. The probabilities enter P V as two bf16 terms (2^-16),
    one (2^-8; `one_term`), or two tf32 terms (2^-22), ex2.approx adds 2^-22 and sums over n keys (n / 16 + 32) 2^-23."""
    T, H, D = q.shape
    group = H // cache.kv_heads
    f32 = cache.k.dtype == torch.float32
    O = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    L = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(O), torch.zeros_like(L).nan_to_num(neginf=0.0)
    bl = torch.zeros(T, H, dtype=torch.float64, device=q.device)
    at = 0
    for b, n in enumerate(new):
        slot = slots[b]
        k, v = gather(cache, slot, plane, layout)
        size = k.shape[0]
        p = torch.arange(size - n, size, device=q.device)
        j = torch.arange(size, device=q.device)
        see = torch.ones(n, size, dtype=torch.bool, device=q.device)
        if causal:
            see &= j[None] <= p[:, None]
        if window:
            see &= j[None] > p[:, None] - window
        for h in range(H):
            kh, vh = k[:, h // group], v[:, h // group]
            qh = q[at:at + n, h].double()
            z = (scale * qh @ kh.T).masked_fill(~see, -math.inf)
            mass = scale * qh.abs() @ kh.abs().T
            e = (mass * (D * 2.0 ** -23 + (2.0 ** -21 if f32 else 0.0))).masked_fill(~see, 0.0)
            e = e.amax(1, keepdim=True) if size else e.sum(1, keepdim=True)
            lse = torch.logsumexp(z, 1) if size else torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
            w = torch.where(see, torch.exp(z - lse.nan_to_num(neginf=0.0)[:, None]), 0.0)
            O[at:at + n, h] = w @ vh
            L[at:at + n, h] = lse
            up = 2.0 ** -22 if f32 else 2.0 ** -8 if one_term else 2.0 ** -16
            up += (size / 16 + 32) * 2.0 ** -23
            bo[at:at + n, h] = (2 * e + up) * (w @ vh.abs())
            bl[at:at + n, h] = e[:, 0] + (size / 16 + 32) * 2.0 ** -23 + lse.nan_to_num(neginf=0.0).abs() * 2.0 ** -22
        at += n
    return O, L, bo, bl


def freqs(rot, base, s):
    """Frequencies (radians a token) and mscale, pair by pair from the formulas."""
    s = s or {"kind": "none"}
    out = []
    if s["kind"] == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if s["kind"] == "linear":
            f /= s["factor"]
        elif s["kind"] == "bands":
            t = s["original"] * f / (2 * math.pi)
            if t <= s["low"]:
                f /= s["factor"]
            elif t < s["high"]:
                w = (t - s["low"]) / (s["high"] - s["low"])
                f = (1 - w) * f / s["factor"] + w * f
        elif s["kind"] == "yarn":
            def edge(beta):
                return rot * math.log(s["original"] / (2 * math.pi * beta)) / (2 * math.log(base))
            a, b = max(math.floor(edge(s["beta_fast"])), 0), min(math.ceil(edge(s["beta_slow"])), rot - 1)
            g = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = g * f / s["factor"] + (1 - g) * f
        out.append(f)
    return out, (0.1 * math.log(s["factor"]) + 1.0 if s["kind"] == "yarn" else 1.0)


def rotate(x, pos, rot, base, scaling, layout, inverse=False):
    """x [T, heads, D] fp64 rotated, and a bound on the kernel's error before the output's rounding: cos and sin to 8
    units of 2^-24 (sincospif's 2, the angle's remainder to 2^-24 of an eighth turn, mscale's rounding), three fp32
    operations, and the frequencies' own 2^-50 (of angles up to pos * f)."""
    f, m = freqs(rot, base, scaling)
    x = x.double()
    a = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = (a.cos() * m)[:, None], (a.sin() * (-m if inverse else m))[:, None]
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    e = (x[..., i].abs() + x[..., j].abs()) * m * (12 * 2.0 ** -24 + a.abs()[:, None] * 2.0 ** -50)
    bound[..., i] = e
    bound[..., j] = e
    return y, bound


def close(got, ref, bound, what):
    """|got - ref| within `bound` plus the rounding of got's type."""
    d = (got.double() - ref).abs()
    lim = bound + U[got.dtype] * (ref.abs() + bound) + 1e-38
    bad = ~(d <= lim)
    assert not bool(bad.any()), (what, int(bad.sum()), float((d / lim).nan_to_num(nan=math.inf).max()))


class Model:
    """The page operations on Python lists, as include/fakv.h words them."""

    def __init__(self, cache):
        self.page, self.max_pages = cache.page_size, cache.table.shape[1]
        self.lens = cache.lens.tolist()
        self.rows = [[p for p in r if p >= 0] for r in cache.table.tolist()]
        self.refs = cache.refs.tolist()
        self.k, self.v = cache.k.clone(), cache.v.clone()
        self.bits = 0

    def need(self, n):
        return -(-n // self.page)

    def grow(self, slots, add):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        refs0, seen, used, asked, drops = list(self.refs), set(), 0, 0, []
        for s, a in zip(slots, add):
            if not 0 <= s < len(self.lens):
                self.bits |= 2
                continue
            if s in seen:
                self.bits |= 4
                continue
            seen.add(s)
            n = self.lens[s]
            if a < 0:
                self.bits |= 32
                continue
            if n + a > self.max_pages * self.page:
                self.bits |= 8
                continue
            copy = a > 0 and n % self.page != 0 and refs0[self.rows[s][n // self.page]] > 1
            want = self.need(n + a) - self.need(n) + copy
            asked += want
            if want and asked > len(free):
                self.bits |= 1
                continue
            mine = free[used:used + want]
            used += want
            for p in mine:
                self.refs[p] = 1
            if copy:
                old = self.rows[s][-1]
                drops.append(old)
                self.rows[s][-1] = mine[0]
                self.k[:, mine[0]], self.v[:, mine[0]] = self.k[:, old], self.v[:, old]
                mine = mine[1:]
            self.rows[s] += mine
            self.lens[s] += a
        for p in drops:
            self.refs[p] -= 1

    def fork(self, src, dst):
        rows, lens, todo = [list(r) for r in self.rows], list(self.lens), []
        for s, d in zip(src, dst):
            if not 0 <= d < len(lens):
                self.bits |= 2
            elif d in [x[1] for x in todo]:
                self.bits |= 4
            elif not 0 <= s < len(lens):
                self.bits |= 2
                todo.append((None, d))
            else:
                todo.append((s, d))
        for s, d in todo:
            if s is not None:
                for p in rows[s]:
                    self.refs[p] += 1
        for s, d in todo:
            if s is not None:
                for p in rows[d]:
                    self.refs[p] -= 1
                self.rows[d], self.lens[d] = list(rows[s]), lens[s]

    def free(self, slots, keep=None):
        seen = set()
        for i, s in enumerate(slots):
            if not 0 <= s < len(self.lens):
                self.bits |= 2
                continue
            if s in seen:
                self.bits |= 4
                continue
            seen.add(s)
            k = 0 if keep is None else keep[i]
            if k < 0:
                self.bits |= 32
                k = 0
            self.lens[s] = min(self.lens[s], k)
            for p in self.rows[s][self.need(self.lens[s]):]:
                self.refs[p] -= 1
            self.rows[s] = self.rows[s][:self.need(self.lens[s])]

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]

    def same(self, cache, what):
        assert cache.lens.tolist() == self.lens, what
        got = cache.table.tolist()
        want = [r + [-1] * (self.max_pages - len(r)) for r in self.rows]
        assert got == want, what
        assert cache.refs.tolist() == self.refs, what
        for x, y in ((cache.k, self.k), (cache.v, self.v)):
            live = torch.tensor([r > 0 for r in self.refs], device=x.device)
            assert torch.equal(x[:, live].nan_to_num(nan=77.0), y[:, live].nan_to_num(nan=77.0)), what
        assert int(cache.status.item()) == self.bits, (what, int(cache.status.item()), self.bits)
