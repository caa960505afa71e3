"""GPU checks that the page calls leave out what they refuse: an entry with a slot, a length, a count or a page that
is not one leaves lens, table and refs as they were and sets its status bit, and the entries beside it are served."""
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


def vec(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def state(cache):
    return [x.tolist() for x in (cache.lens, cache.table, cache.refs)]


def bits(kv, cache):
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    return e.value.bits


BAD = [-1, -(1 << 31), 9 * 8 + 1, (1 << 31) - 1]  # no length of a row of 9 pages of 8 tokens


def small(kv):
    return ref.make_cache(kv, [20, 9, 30, 16], 8, 1, 16, BF, max_pages=9, extra=8)


@pytest.mark.parametrize("length", BAD)
def test_grow_leaves_out_a_bad_length(kv, length):
    cache = small(kv)
    cache.lens[1] = length
    m = ref.Model(cache)
    cache.grow(vec(0, 1, 2), vec(5, 5, 5))
    m.grow([0, 2], [5, 5])  # (slot 1 asks for nothing)
    m.bits = kv.BAD_LENGTH
    m.same(cache, length)


@pytest.mark.parametrize("page", [-1, 1 << 20, -(1 << 31)])
def test_grow_leaves_out_a_missing_last_page(kv, page):
    cache = small(kv)
    cache.table[1, 1] = page  # slot 1: 9 tokens, the ninth on this page
    before = state(cache)
    cache.grow(vec(1), vec(3))
    assert bits(kv, cache) == kv.BAD_PAGE and state(cache) == before
    cache.grow(vec(1), vec(30))  # (also where new pages would come after it)
    assert bits(kv, cache) == kv.BAD_PAGE and state(cache) == before
    m = ref.Model(cache)
    cache.grow(vec(1, 2, 0), vec(9, 9, 9))  # its neighbours are served, with the lowest pages
    m.grow([2, 0], [9, 9])
    got = state(cache)
    assert got[0] == m.lens and got[2] == m.refs and got[1][1] == before[1][1]
    for s in (0, 2):
        assert [p for p in got[1][s] if p >= 0] == m.rows[s]
    assert bits(kv, cache) == kv.BAD_PAGE
    cache.grow(vec(1), vec(0))  # nothing new, nothing looked at
    cache.check()


# one launch for short lists of short rows, two for the rest
@pytest.mark.parametrize("max_pages", [9, 300])
@pytest.mark.parametrize("who", ["source", "destination"])
@pytest.mark.parametrize("length", [-1, (1 << 31) - 1])
def test_fork_leaves_out_a_bad_length(kv, max_pages, who, length):
    cache = ref.make_cache(kv, [20, 9, 30, 16], 8, 1, 16, BF, max_pages=max_pages)
    m = ref.Model(cache)
    cache.lens[1] = length
    src, dst = ([1, 0], [3, 2]) if who == "source" else ([3, 0], [1, 2])
    cache.fork(vec(*src), vec(*dst))
    m.fork([0], [2])
    m.lens[1], m.bits = length, kv.BAD_LENGTH
    m.same(cache, who)


@pytest.mark.parametrize("length", BAD)
def test_free_leaves_out_a_bad_length(kv, length):
    cache = small(kv)
    cache.lens[1] = length
    m = ref.Model(cache)
    for keep in (None, [4, 4, 4]):
        cache.free(vec(0, 1, 2), None if keep is None else vec(*keep))
        m.free([0, 2], None if keep is None else [4, 4])
        m.bits = kv.BAD_LENGTH
        m.same(cache, (length, keep))
        m.bits = 0
        assert bits(kv, cache) == kv.BAD_LENGTH


def test_free_leaves_out_a_negative_keep(kv):
    cache = small(kv)
    m = ref.Model(cache)
    cache.free(vec(0, 1, 2), vec(3, -1, -(1 << 31)))
    m.free([0], [3])
    m.bits = kv.BAD_LENGTH
    m.same(cache, "keep")
