"""GPU checks of the tensor-core tiles (chunks of a bf16 cache) with pages that are none: numbers out of range are read
as zeros and reported, entries that no row sees are not looked at, rows that see nothing are zeros."""
import pytest
import torch

import _kv_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_fa_fwd_02_gb300 import kv as m
    return m


def cu_of(new):
    return torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("number", [-1, 1 << 20, (1 << 31) - 1, -(1 << 31)])
def test_a_page_number_out_of_range(kv, page, number):
    n, lens = 150, [1300, 700]
    cache = ref.make_cache(kv, lens, page, 2, 64, BF)
    q = randn(2 * n, 8, 64)
    want, want_l = cache.attend(q, cu_of([n, n]))
    col = 300 // page
    lo, hi = col * page, min(1300, (col + 1) * page)
    old = int(cache.table[0, col])
    cache.table[0, col] = number
    o, lse = cache.attend(q, cu_of([n, n]))
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_PAGE
    assert torch.equal(o[n:], want[n:]) and torch.equal(lse[n:], want_l[n:])
    # the page's tokens as zeros
    cache.table[0, col] = old
    cache.k[0, old, :hi - lo], cache.v[0, old, :hi - lo] = 0.0, 0.0
    same, same_l = cache.attend(q, cu_of([n, n]))
    cache.check()
    assert torch.equal(o, same) and torch.equal(lse, same_l)


@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("page", [8, 32, 256])
def test_pages_below_a_window_may_be_gone(kv, n, page):
    window, size = 100, 2000
    cache = ref.make_cache(kv, [size], page, 2, 64, BF)
    q = randn(n, 8, 64)
    want = cache.attend(q, cu_of([n]), window=window)
    first = size - n - window + 1  # the first key that any row sees
    cache.table[0, :first // page] = -1
    got = cache.attend(q, cu_of([n]), window=window)
    cache.check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D", [64, 128])
def test_rows_and_sequences_that_see_nothing(kv, D):
    # a bad length, a bad slot, a sequence with fewer tokens than rows, and an ordinary one between them
    new, order = [200, 130, 300, 140, 290], [0, 1, 2, -5, 3]
    cache = ref.make_cache(kv, [500, 500, 40, 900], 16, 2, D, BF)
    cache.lens[1] = 1 << 30
    T = sum(new)
    q = randn(T, 8, D)
    slots = torch.tensor(order, dtype=torch.int32).cuda()
    o, lse = torch.full((T, 8, D), 9.0, dtype=BF, device="cuda"), torch.full((T, 8), 9.0, device="cuda")
    cache.attend(q, cu_of(new), slots, out=o, lse=lse)
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_LENGTH | kv.BAD_SLOT
    none = torch.zeros(T, dtype=torch.bool)
    none[200:330] = True        # the bad length
    none[330:330 + 260] = True  # positions -260 .. -1 of slot 2
    none[630:770] = True        # the bad slot
    none = none.cuda()
    assert bool((o[none] == 0).all()) and bool(torch.isneginf(lse[none]).all())
    for a, e_, slot in ((0, 200, 0), (590, 630, 2), (770, T, 3)):
        ro, rl, bo, bl = ref.attend(cache, q[a:e_], [e_ - a], [slot], D ** -0.5, True, 0, one_term=True)
        ref.close(o[a:e_], ro, bo, ("O", slot))
        ref.close(lse[a:e_], rl, bl, ("LSE", slot))
