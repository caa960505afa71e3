"""Seeded random calls of attention over the cache in 4 or 8 bits: shapes, masks, types, and K and V whose tokens differ in size by
many powers of two, or are zero, or constant; each batch once or many times in a call, so that items are cut and not cut.
Against bounds that each row's own keys give (_kvq_seen.py)."""
import math
import random

import pytest
import torch

import _kv_ref
import _kvq_ref as ref
import _kvq_seen as seen

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_fa_fwd_02_gb300 import kv as m
    return m


def cu_of(new):
    return torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("seed", range(64))
def test_random_calls(kv, seed):
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    D, bits, group = rng.choice(ref.SHAPES)
    dtype, odt = rng.choice([BF, BF, F32]), rng.choice([BF, F32])
    B, rep, HKV = rng.choice([1, 1, 2, 5]), rng.choice([1, 2, 3, 4, 7]), rng.choice([1, 2])
    new = [rng.choice([0, 1, 2, 5, 20, 60, 130] if B > 1 else [1, 3, 9, 40, 150]) for _ in range(B)]
    new[0] = max(1, new[0])
    lens = [max(0, n + rng.choice([0, 0, 5, 100, 700, -3])) for n in new]
    causal, window, many = rng.random() < 0.7, rng.choice([0, 0, 1, 17, 100]), rng.choice([1, 40, 150])
    cache, _ = ref.make(kv, lens, rng.choice([8, 16, 64, 256]), HKV, D, bits, group, dtype, seed=seed, stored=False)
    T, rows = sum(lens), sum(new)

    def tokens(spans):
        e = torch.randn(T, 1, 1, generator=g) * rng.choice(spans)
        if rng.random() < 0.5:  # a few tokens of another size
            e = e * (torch.rand(T, 1, 1, generator=g) < 0.05)
        x = torch.randn(T, HKV, D, generator=g) * 2.0 ** e.round().clamp(-60, 60)
        if rng.random() < 0.3:
            x[torch.rand(T, generator=g) < 0.1] = rng.choice([0.0, 1.5])
        return x.to(dtype).cuda()

    if T:
        cache.append(None, tokens([0, 1, 3, 8]), tokens([0, 2, 10, 25]), cu_of(lens))
    q = (torch.randn(rows, HKV * rep, D, generator=g) * rng.choice([0.3, 1.0, 4.0])).to(dtype).cuda()
    slots = torch.arange(B, dtype=torch.int32).repeat(many).cuda()
    o, l = cache.attend(q.repeat(many, 1, 1), cu_of(new * many), slots, causal=causal, window=window, out_dtype=odt)
    cache.check()
    tiles = dtype == BF and rows * rep > (48 if D > 64 else 64) * B
    want, want_l, bo, bl = seen.attend(cache, q, new, list(range(B)), D ** -0.5, causal, window, 0, tiles, odt == F32)
    o, l = o.cpu().unflatten(0, (many, rows)), l.cpu().unflatten(0, (many, rows))
    _kv_ref.close(o, want, bo, "O")
    none = want_l == -math.inf
    assert torch.equal(l == -math.inf, none.expand_as(l)) and bool((o[none.expand_as(l)] == 0).all())
    assert bool(((l.double() - want_l).abs() <= bl)[~none.expand_as(l)].all())
