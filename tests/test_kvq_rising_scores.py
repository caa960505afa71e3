"""Chunks over the cache in 4 or 8 bits whose rows' references move again and again: scores that rise in both halves of a
tile's keys, V's size that grows in the same tile. What was summed up before has to follow each move."""
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


def rising(kv, bits, n, score, value, rows, H=2, D=128, seed=0, zero=((256, None),)):
    """A cache of one sequence, two groups of V's columns, and queries whose scores of key j are about score[j] (log2); V is
    `value[j]` in size in the second group, and about 1 in the first one, or zero (ranges of keys)."""
    g = torch.Generator().manual_seed(seed)
    cache, _ = ref.make(kv, [n], 16, 1, D, bits, 64, BF, stored=False)
    way = torch.randn(D, generator=g).sign()
    k = score[:, None] * way * (1 + 0.05 * torch.rand(n, D, generator=g)) / D
    v = torch.randn(n, D, generator=g)
    for a, b in zero:
        v[a:b, :64] = 0.0
    v[:, 64:] *= value[:, None]
    cache.append(None, k[:, None].to(BF).cuda(), v[:, None].to(BF).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    q = (way * (1 + 0.02 * torch.randn(rows, H, D, generator=g))).to(BF).cuda()
    return cache, q, 0.6931471805599453  # (of which a score's log2 is the product of q and k)


def check(cache, q, scale, causal, out_dtype):
    """The same sequence and queries 320 times in one call: more items than CTAs, so that many are not shared out tile by
    tile (one whose tiles have a CTA each never moves a reference)."""
    rows, B = q.shape[0], 320
    o, l = cache.attend(q.repeat(B, 1, 1), torch.arange(B + 1, dtype=torch.int32).cuda() * rows,
                        torch.zeros(B, dtype=torch.int32).cuda(), scale=scale, causal=causal, out_dtype=out_dtype)
    cache.check()
    want, want_l, bo, bl = seen.attend(cache, q, [rows], [0], scale, causal, 0, 0, True, out_dtype == F32)
    o, l = o.cpu().unflatten(0, (B, rows)), l.cpu().unflatten(0, (B, rows))
    _kv_ref.close(o, want, bo, "O")
    assert bool(((l.double() - want_l).abs() <= bl).all())


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("grown", [0, 8])
def test_references_that_move_in_both_halves_of_a_tile(kv, bits, causal, grown, out_dtype):
    """From the third tile on scores rise by 2^10 (more than the 2^8 that a reference waits for) with each half, and V by
    2^grown with each tile: O is rescaled twice, or three times, to a tile. The first group's columns are made of the first two
    tiles' keys alone: of them a factor that was lost would be all that is left."""
    n, rows = 128 * 5, 60
    half, tile = torch.arange(n) // 64, torch.arange(n) // 128
    cache, q, scale = rising(kv, bits, n, 10.0 * (half - 3).clamp(min=0).float(), 2.0 ** (grown * (tile - 1).clamp(min=0)), rows)
    check(cache, q, scale, causal, out_dtype)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("bits", [4, 8])
def test_what_the_first_half_of_a_tile_is_beside_one_key_of_the_second(kv, bits, out_dtype):
    """64 keys whose probabilities fall by 2^26 when the tile's second half is looked at: 2^-18 each, and V of the first group's
    columns is 0 everywhere else, so that they are all that these columns are made of."""
    n, rows = 128 * 3, 60
    score = torch.zeros(n)
    score[128:256], score[200], score[256:] = 7.5, 24.6, -20.0
    cache, q, scale = rising(kv, bits, n, score, torch.ones(n), rows, zero=[(0, 128), (192, n)])
    check(cache, q, scale, False, out_dtype)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("down", [16, 22, 28])
def test_keys_of_small_probability_whose_values_are_the_largest(kv, bits, down):
    """A product of a probability and V is lost below 2^-30 of the largest V: 127 keys of 2^-down each beside one."""
    n, rows = 128, 60
    score = torch.zeros(n)
    score[77] = float(down)
    cache, q, scale = rising(kv, bits, n, score, torch.ones(n), rows, zero=[(77, 78)])
    check(cache, q, scale, False, F32)
