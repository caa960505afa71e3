"""Plain references of the cache in 4 or 8 bits: the format by its definition, fp64 arithmetic, and bounds on what the
kernels' arithmetic may add."""
import math

import torch

SHAPES = [  # head_dim, bits, group
    (128, 4, 64), (128, 8, 128), (128, 4, 128), (128, 8, 64), (64, 4, 64), (64, 8, 64), (16, 4, 16), (32, 8, 32),
    (48, 4, 48), (80, 8, 80), (80, 4, 80), (96, 4, 96), (112, 8, 112)]


def down(x):
    """The largest bf16 <= x, fp32."""
    y = x.to(torch.bfloat16)
    over = y.float() > x
    return torch.where(over, torch.nextafter(y, torch.full_like(y, -math.inf)), y).float()


def quantise(x, bits, group):
    """Codes [..., D], scales and offsets [..., groups] of fp32 x, by the definition (IEEE fp32 on the CPU)."""
    x = x.float().cpu().unflatten(-1, (-1, group))
    steps = torch.tensor(2.0 ** bits - 1)
    z = down(x.amin(-1))
    s = -down(-((x.amax(-1) - z) / steps))
    c = torch.round((x - z[..., None]) / s[..., None]).clamp(0, 2 ** bits - 1)
    c = torch.where(s[..., None] > 0, c, 0.0).to(torch.int64)
    bad = ~(x.abs() < 2.0 ** 126).all(-1)
    return c.flatten(-2), s.masked_fill(bad, math.nan), z.masked_fill(bad, math.nan), bad


def tokens(codes, page, chunks, bits, is_v):
    """The code bytes of blocks [pages, heads, bytes], token by token: [pages, heads, page, chunks * 16]."""
    P = codes.shape[0]
    if is_v:
        part = 2 if bits == 4 else 1  # bytes of one of two tokens in turn
        x = codes.reshape(P, -1, page // 8, chunks, 4, 16 // part, 2, part)
        x = x.permute(0, 1, 2, 4, 6, 3, 5, 7)  # octet, pair, token, chunk, pieces
    else:
        x = codes.reshape(P, -1, page // 8, chunks, 8, 16).transpose(3, 4)
    return x.reshape(P, -1, page, chunks * 16)


def unpack(cache, plane=0):
    """What the pages' memory holds: for K and V codes [pages, page, HKV, D], scales and offsets [.., groups]."""
    out = []
    P, S, D, bits, ng = cache.k.shape[1], cache.page_size, cache.head_dim, cache.bits, cache.head_dim // cache.group
    chunks = -(-D * bits // 128)
    for x, is_v in ((cache.k, False), (cache.v, True)):
        b = x[plane].cpu()  # [pages, heads, bytes]
        codes = tokens(b[..., :S * chunks * 16], S, chunks, bits, is_v)
        if bits == 4:
            codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        words = b[..., S * chunks * 16:].reshape(P, -1, S, ng, 2, 2).contiguous().view(torch.int16)[..., 0].contiguous()
        params = words.view(torch.bfloat16).float()
        out.append((codes[..., :D].to(torch.int64).transpose(1, 2), params[..., 0].transpose(1, 2), params[..., 1].transpose(1, 2)))
    return out


def make(kv, lens, page, HKV, D, bits, group, dtype, seed=0, planes=1, slots=None, order=None, extra=3, max_pages=None,
         fill=1.5, stored=True, poison=True, shift=0.0):
    """A QuantCache whose slot order[b] (default b) holds lens[b] random tokens in every plane, its pages in a random
    order; params of tokens that are not there NaN, their codes anything. Returns it and what was appended,
    [plane] -> (k, v) of all tokens in order."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    slots = slots or B
    order = list(range(B)) if order is None else order
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    perm = torch.randperm(pages, generator=g).tolist()
    width = max_pages or max(need + [1]) + 1
    cache = kv.QuantCache.create(planes, pages, page, HKV, D, slots, width, bits, group, dtype)
    if poison:
        for x in (cache.k, cache.v):
            x.copy_(torch.randint(0, 256, x.shape, generator=g, dtype=torch.uint8))
            codes = page * (-(-D * bits // 128)) * 16
            x[..., codes:] = 255  # s = z = NaN
    at = 0
    for b, n in enumerate(lens):
        mine = perm[at:at + need[b]]
        at += need[b]
        cache.table[order[b], :need[b]] = torch.tensor(mine, dtype=torch.int32)
        cache.lens[order[b]] = n
        cache.refs[torch.tensor(mine, dtype=torch.long)] = 1
    T, given = sum(lens), []
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()
    where = torch.tensor(order, dtype=torch.int32).cuda()
    for l in range(planes if stored else 0):
        k = ((torch.randn(T, HKV, D, generator=g) + shift) * fill).to(dtype).cuda()
        v = (torch.randn(T, HKV, D, generator=g) + shift).to(dtype).cuda()
        cache.append(None, k, v, cu, where, layer=l)
        given.append((k, v))
    return cache, given


def held(cache, slot, plane=0):
    """For K and V of a slot's tokens, fp64: values [len, HKV, D], and (scale, offset) by column."""
    n, page = int(cache.lens[slot]), cache.page_size
    rows = cache.table[slot, :-(-n // page)].long().cpu()
    out = []
    for codes, s, z in unpack(cache, plane):
        c = codes[rows].flatten(0, 1)[:n].double()
        s, z = (t[rows].flatten(0, 1)[:n].double().repeat_interleave(cache.group, -1) for t in (s, z))
        out.append((s * c + z, s, z, c))
    return out


def attend(cache, q, new, slots, scale, causal, window, plane=0, tiles=False, out_f32=None):
    """O, LSE of the rows (fp64, on the CPU), and bounds on |O - ref| (before the output's rounding) and |LSE - ref|.

    Few rows. q enters as fp16 times a power of two (2^-35 of its row's largest is lost), fp32 q in two terms (2^-22). A
    product with codes of D columns takes D / 16 steps of the tensor cores (for each term), each of which cuts off at
    2^-23 of a partial sum twice at most: the partial sums are at most m = sum |q| c. Where O is fp32
    they are centred codes x: m = sum |q| |x|. A score is s m 2^-23 (D / 8 + 2) (times the terms) off from that, and
    two fused operations a group, below 4 * 2^-24 of s m + |z| sum |q|. A score error e moves its probability by the
    factor exp(e): O_d by at most 2 e A_d, A_d = sum_j p_j |v_jd|, the LSE by e. Probabilities times scales enter as one
    fp16 term (2^-11; O in bf16) or two (2^-22) of s x, and what lies under 2^-30 of the largest scale s' is lost (n keys,
    the sum of probabilities being at least 1 as they are taken); p z' in fp32; ex2.approx adds 2^-22; sums over n keys
    (n / 16 + 32) 2^-23 and, for the offsets, n 2^-24, each of M_d = sum_j p_j (s |x| + |z'|).

    Many rows (`tiles`): q as above; K is x s (nibbles: exact in fp16, but for 2^-25 of 2^-4 of the largest of 32 keys) and
    z' in two terms (2^-22 of it, and of q's sum, which is two terms too); 8 bits take a second plane of as many steps. V
    and P are rounded to fp16 (half a step 2^-11): V after x s + z', s and z' rounded too, so it is off by at most 2^-11 of
    s |x| + |z'| and by 2^-32 of the largest."""
    T, H, D = q.shape
    f32 = q.dtype == torch.float32
    q = q.double().cpu()
    rep = H // cache.kv_heads
    mid = 8.0 if cache.bits == 4 else 128.0
    out_f32 = f32 if out_f32 is None else out_f32
    terms = 2 if f32 else 1
    O = torch.zeros(T, H, D, dtype=torch.float64)
    L = torch.full((T, H), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(O), torch.zeros(T, H, dtype=torch.float64)
    at = 0
    for b, n in enumerate(new):
        (k, ks, kz, kc), (v, vs, vz, vc) = held(cache, slots[b], plane)
        size = k.shape[0]
        p = torch.arange(size - n, size)
        j = torch.arange(size)
        see = torch.ones(n, size, dtype=torch.bool)
        if causal:
            see &= j[None] <= p[:, None]
        if window:
            see &= j[None] > p[:, None] - window
        for h in range(H):
            i = h // rep
            qh, qa = q[at:at + n, h], q[at:at + n, h].abs()
            if not size:
                continue
            z = (scale * qh @ k[:, i].T).masked_fill(~see, -math.inf)
            if tiles:
                size_k = (ks * (kc - mid).abs() + (kz + mid * ks).abs() + ks * mid)[:, i]
                m = qa @ size_k.T
                e = scale * (m * ((D / 4 + 4) * 2.0 ** -23 + 2.0 ** -21) + size_k.max() * 2.0 ** -29 * qa.sum(1, keepdim=True)
                             + qa.amax(1, keepdim=True) * 2.0 ** -35 * size_k.sum(1))
            else:
                sizes = ks * ((kc - mid).abs() if out_f32 else kc)
                m = qa @ sizes[:, i].T
                e = scale * (terms * (D / 8 + 2) * 2.0 ** -23 * m + 2.0 ** -22 * (m + qa @ (kz.abs() + mid * ks)[:, i].T)
                             + qa.amax(1, keepdim=True) * 2.0 ** -35 * (ks * (kc + mid))[:, i].sum(1))
                if f32:
                    e = e + scale * 2.0 ** -22 * (qa @ (k[:, i].abs() + ks[:, i] * mid).T)
            e = e.masked_fill(~see, 0.0).amax(1, keepdim=True)
            lse = torch.logsumexp(z, 1)
            w = torch.where(see, torch.exp(z - lse.nan_to_num(neginf=0.0)[:, None]), 0.0)
            O[at:at + n, h] = w @ v[:, i]
            L[at:at + n, h] = lse
            mass = vs * (vc - mid).abs() + (vz + mid * vs).abs()
            up = (2.0 ** -22 if out_f32 else 2.0 ** -11) + 2.0 ** -22 + (size / 16 + 32) * 2.0 ** -23 + size * 2.0 ** -24
            if tiles:
                up += 2.0 ** -11 + 2.0 ** -11
            lost = size * 2.0 ** -30 * float(vs[:, i].max()) * mid
            bo[at:at + n, h] = 2 * e * (w @ v[:, i].abs()) + up * (w @ mass[:, i]) + lost
            if tiles:
                bo[at:at + n, h] += size * 2.0 ** -30 * mass[:, i].max()
            bl[at:at + n, h] = e[:, 0] + (size / 16 + 32) * 2.0 ** -23 + lse.nan_to_num(neginf=0.0).abs() * 2.0 ** -22
        at += n
    return O, L, bo, bl
