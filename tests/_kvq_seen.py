"""Attention over the cache in 4 or 8 bits in 64 bits, and bounds on what the kernels' arithmetic may add that are made of
what a row SEES: the keys that its mask hides have no part in them, and what a product loses is against the largest scores
and values of the row's keys up to it. (_kvq_ref.attend's are against the largest of all keys.)

A score of key j, few rows: q as fp16 (2^-35 of its row's largest is lost; fp32 in two terms, 2^-22), exact codes, D / 16
steps of the tensor cores for each term, each cut off at 2^-23 of a partial sum twice at most, and a few fp32 operations:
e_j = scale (terms (D / 8 + 2) 2^-23 m_j + 2^-22 (m_j + |z'| sum |q|)), m_j = sum |q| s c. Many rows: twice the steps; K's
scales exact in fp16 or to 2^-21 of the key's own size, offsets and sums of q in two terms (2^-22 each): with m_j = sum |q| (s |x| +
|z'| + s mid), e_j = scale m_j ((D / 4 + 4) 2^-23 + 2^-20).

A score error e moves a probability by exp(e), O by 2 e A with A = sum w |v - O| (e up to 1/4; beyond that O is some mean of
the V that may have a weight, unless that is one key's alone), the LSE by e: the largest e_j of the keys that may have a
weight. Those whose score, with its error, is 50 and more below what the largest one's is at least have none, and n e^-50 of
the largest value is added for them.

A product of a probability and V, few rows: probability times scale in fp16 (one term 2^-11, two 2^-22), of which what is under
2^-30 of the largest scale S so far is lost, taken against the largest score so far: 2^-30 |x| S exp(top - LSE) of a code x
(of a scale that is not 0). Many rows: V to 2^-11 twice (z', then s x + z'), P to 2^-11, and P's floor in fp16, at most three
roundings of 2^-25, P being p 2^(E - R): E the exponent that brings the key's largest value U below 2^7 (so 2^-E < 2^7 / U), R
at most 5 less than that of the largest value V so far (2^R <= 2^-11 V), or up to 3 more (of a neighbour that is hidden): 2^-23
2^(R - E) of a value v, and 2 for a reference that is a whole power of two: 2^-23 V |v| / U exp(top - LSE). A group of keys that is gone
through at once has 128 (few rows: up to 64) of them; a part that begins later has seen less, and smaller."""
import math

import torch

import _kvq_ref as ref


def attend(cache, q, new, slots, scale, causal=True, window=0, plane=0, tiles=False, out_f32=None):
    """O, LSE (fp64, on the CPU) and bounds on |O - ref| (before the output's rounding) and |LSE - ref|."""
    T, H, D = q.shape
    f32 = q.dtype == torch.float32
    q = q.double().cpu()
    rep, bits = H // cache.kv_heads, cache.bits
    mid, steps = (8.0, 15.0) if bits == 4 else (128.0, 255.0)
    out_f32 = f32 if out_f32 is None else out_f32
    terms, step = (2 if f32 else 1), (128 if tiles else 64)
    O = torch.zeros(T, H, D, dtype=torch.float64)
    L = torch.full((T, H), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(O), torch.zeros(T, H, dtype=torch.float64)
    at = 0
    for b, n in enumerate(new):
        (k, ks, kz, kc), (v, vs, vz, vc) = ref.held(cache, slots[b], plane)
        size = k.shape[0]
        if not size or not n:
            at += n
            continue
        p, j = torch.arange(size - n, size), torch.arange(size)
        see = torch.ones(n, size, dtype=torch.bool)
        if causal:
            see &= j[None] <= p[:, None]
        if window:
            see &= j[None] > p[:, None] - window

        def so_far(x):  # [n, size]: the largest of the row's keys up to the end of each one's step
            x = torch.nn.functional.pad(x, (0, -size % step), value=-math.inf).unflatten(1, (-1, step)).amax(-1)
            return torch.cummax(x, 1)[0].repeat_interleave(step, 1)[:, :size]

        for h in range(H):
            i = h // rep
            qh, qa = q[at:at + n, h], q[at:at + n, h].abs()
            z = (scale * qh @ k[:, i].T).masked_fill(~see, -math.inf)
            if tiles:
                m = qa @ (ks * (kc - mid).abs() + (kz + mid * ks).abs() + ks * mid)[:, i].T
                e = scale * (m * ((D / 4 + 4) * 2.0 ** -23 + 2.0 ** -20) + qa.amax(1, keepdim=True) * 2.0 ** -35 * (
                    ks * (kc + mid) + kz.abs())[:, i].sum(1))
            else:
                m = qa @ (ks * ((kc - mid).abs() if out_f32 else kc))[:, i].T
                e = scale * (terms * (D / 8 + 2) * 2.0 ** -23 * m + 2.0 ** -22 * (m + qa @ (kz.abs() + mid * ks)[:, i].T)
                             + qa.amax(1, keepdim=True) * 2.0 ** -35 * (ks * (kc + mid))[:, i].sum(1))
                if f32:
                    e = e + scale * 2.0 ** -22 * (qa @ (k[:, i].abs() + ks[:, i] * mid).T)
            lse = torch.logsumexp(z, 1)
            base = lse.nan_to_num(neginf=0.0)[:, None]
            w = torch.where(see, torch.exp(z - base), 0.0)
            may = see & (z + e > (z - e).amax(1, keepdim=True) - 50.0)
            e = torch.where(may, e, 0.0).amax(1, keepdim=True)
            several = (may.sum(1, keepdim=True) > 1) & (e > 0.25)
            O[at:at + n, h] = w @ v[:, i]
            L[at:at + n, h] = lse
            mass = (vs * (vc - mid).abs() + (vz + mid * vs).abs())[:, i]
            seen = lambda x: torch.where(see, x[None], 0.0)  # noqa: E731
            top = torch.exp(so_far(z) - base)
            up = 3 * 2.0 ** -11 if tiles else 2.0 ** -22 if out_f32 else 2.0 ** -11
            up += 2.0 ** -22 + (size / 16 + 32) * 2.0 ** -23 + size * 2.0 ** -24
            size_v = (torch.maximum(vz.abs(), (vs * steps + vz).abs()) if tiles else vs)[:, i].amax(1)
            largest = so_far(seen(size_v)) * top * see
            if tiles:
                floor = 2.0 ** -23 * (largest / size_v.clamp(min=1e-100)) @ mass
            else:
                floor = 2.0 ** -30 * largest @ ((vc - mid).abs() * (vs > 0))[:, i]
            moved = torch.stack([(w[r, :, None] * (v[:, i] - O[at + r, h]).abs()).sum(0) for r in range(n)])
            moved = torch.where(several, 2 * seen(v[:, i].abs().amax(1)).amax(1, keepdim=True), 2 * e * moved)
            none = size * math.exp(-50.0) * seen(mass.amax(1)).amax(1, keepdim=True)
            bo[at:at + n, h] = moved + up * (w @ mass) + floor + none
            bl[at:at + n, h] = e[:, 0] + (size / 16 + 32) * 2.0 ** -23 + lse.nan_to_num(neginf=0.0).abs() * 2.0 ** -22
        at += n
    return O, L, bo, bl
