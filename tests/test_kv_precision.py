"""GPU checks of accuracy at the bounds of the arithmetic that each path uses (tests/_kv_ref.py derives them): fp32
outputs of the tensor-core tiles, decoding and drafts with two-term probabilities, padded batches, and fp32 caches
through a whole step."""
import math

import pytest
import torch

import _kv_ref as ref

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


def randn(*shape, dtype=F32, seed=0, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * mul).to(dtype).cuda()


@pytest.mark.parametrize("new,lens,H,HKV,D,page,causal,window", [
    ([200], [3000], 8, 1, 64, 8, True, 0),
    ([33, 1, 129], [33, 500, 2000], 10, 2, 128, 16, True, 0),
    ([300, 2], [300, 9000], 4, 4, 80, 256, True, 500),
    ([70], [700], 6, 2, 32, 64, False, 0),
    ([260], [260], 32, 1, 128, 16, True, 0)])
def test_fp32_outputs_of_chunks(kv, new, lens, H, HKV, D, page, causal, window):
    """Many rows per sequence of a bf16 cache: an fp32 O has its probabilities in two bf16 terms, LSE is the same."""
    cache = ref.make_cache(kv, lens, page, HKV, D, BF, seed=3)
    q = randn(sum(new), H, D, dtype=BF, seed=4, mul=1.5)
    assert sum(new) * (H // HKV) > 16 * len(new)
    o, lse = cache.attend(q, cu_of(new), None, 0.11, causal, window, out_dtype=F32)
    cache.check()
    ro, rl, bo, bl = ref.attend(cache, q, new, list(range(len(new))), 0.11, causal, window)
    ref.close(o, ro, bo, "O")
    ref.close(lse, rl, bl, "LSE")


@pytest.mark.parametrize("new,lens", [([3, 1], [50, 333]), ([1, 1], [300, 111]), ([1], [300]), ([4] * 3, [900, 4, 77])])
def test_few_rows_have_two_terms(kv, new, lens):
    cache = ref.make_cache(kv, lens, 16, 2, 64, BF, planes=3)
    q = randn(sum(new), 12, 64, dtype=BF, seed=5)[:, :8]  # a slice of a projection of q, k and v
    assert sum(new) * 4 <= 16 * len(new)
    for plane in range(3):
        for odt in (BF, F32):
            o, lse = cache.attend(q, cu_of(new), layer=plane, out_dtype=odt)
            ro, rl, bo, bl = ref.attend(cache, q, new, list(range(len(new))), 0.125, True, 0, plane)
            ref.close(o, ro, bo, "O")
            ref.close(lse, rl, bl, "LSE")


@pytest.mark.parametrize("pad", [3, 40, 500])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_padded_batch_is_the_batch(kv, dtype, pad):
    """Rows behind the last sequence count where the kernel is chosen, never in what the others get."""
    lens = [700, 33, 1, 2000, 5, 64, 900, 17]
    cache = ref.make_cache(kv, lens, 16, 2, 64, dtype)
    q = randn(8 + pad, 8, 64, dtype=dtype, seed=6)
    q[8:] = float("nan")
    ro, rl, bo, bl = ref.attend(cache, q[:8], [1] * 8, list(range(8)), 0.125, True, 0)
    for odt in (F32, BF):
        one = dtype == BF and odt == BF and (8 + pad) * 4 > 16 * 8
        b2 = ref.attend(cache, q[:8], [1] * 8, list(range(8)), 0.125, True, 0, one_term=True)[2] if one else bo
        o, lse = torch.full((8 + pad, 8, 64), 9.0, dtype=odt, device="cuda"), torch.full((8 + pad, 8), 9.0, device="cuda")
        cache.attend(q, cu_of([1] * 8), out=o, lse=lse)
        cache.check()
        ref.close(o[:8], ro, b2, "O")
        ref.close(lse[:8], rl, bl, "LSE")
        assert bool((o[8:] == 9.0).all()) and bool((lse[8:] == 9.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [(37, 12), (6, 9, 1)])
def test_a_prompt_and_its_next_tokens(kv, dtype, chunks):
    """grow, append and attend of a prompt in parts and then token by token, each O within the bound of its arithmetic
    over what was appended, which is bit for bit what rope.apply makes of the keys."""
    H, HKV, D, page = 4, 2, 64, 16
    cache = kv.PagedCache.create(1, 12, page, HKV, D, 2, 8, dtype)
    rope = kv.Rope(D, base=500000.0)
    ks, vs, at = [], [], 0
    for i, n in enumerate(chunks + (1, 1, 3)):
        q, k, v = (randn(n, h, D, dtype=dtype, seed=10 * i + j) for j, h in enumerate((H, HKV, HKV)))
        slot, cu = torch.tensor([1], dtype=torch.int32).cuda(), cu_of([n])
        cache.grow(slot, torch.tensor([n], dtype=torch.int32).cuda())
        r = cache.append(q, k, v, cu, slot, rope)
        o, lse = cache.attend(r, cu, slot)
        pos = torch.arange(at, at + n).cuda()
        at += n
        assert torch.equal(r, rope.apply(q, None, pos)[0])
        ks.append(rope.apply(k, None, pos)[0])
        vs.append(v)
        for got, want in zip(ref.gather(cache, 1), (ks, vs)):
            assert torch.equal(got, torch.cat(want).double())
        one = dtype == BF and n * 2 > 16
        ro, rl, bo, bl = ref.attend(cache, r, [n], [1], D ** -0.5, True, 0, one_term=one)
        ref.close(o, ro, bo, ("O", i))
        ref.close(lse, rl, bl, ("LSE", i))
    cache.check()
