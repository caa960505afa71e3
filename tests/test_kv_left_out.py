"""GPU checks that the page calls leave out what they refuse: an entry with a slot, a length, a count or a page that
is not one leaves lens, table and refs as they were and sets its status bit, and the entries beside it are served."""
import random

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


def test_compact_leaves_rows_of_bad_lengths_in_place(kv):
    # their pages are counted and move with the others
    cache = small(kv)
    m = ref.Model(cache)
    m.free([0, 2])
    cache.free(vec(0, 2))
    cache.lens[1], cache.lens[3] = -3, 1 << 30
    m.compact()
    cache.compact()
    m.lens[1], m.lens[3] = -3, 1 << 30
    m.same(cache, "compact")


def test_compact_renumbers_whole_rows(kv):
    """Entries past a row's length (a length lowered by hand, pages in reserve) go on naming the page they named."""
    cache = ref.make_cache(kv, [40, 70, 64, 33], 8, 1, 16, BF)
    held = [[int(p) for p in r if p >= 0] for r in cache.table.tolist()]
    k0 = cache.k.clone()
    cache.free(vec(0))
    cache.lens[1] = 17   # of 9 pages, 3 by its length
    cache.lens[3] = 0
    cache.compact()
    cache.check()
    rows = cache.table.tolist()
    assert rows[0] == [-1] * len(rows[0])
    live = int((cache.refs > 0).sum())
    assert bool((cache.refs[:live] == 1).all()) and bool((cache.refs[live:] == 0).all())
    seen = []
    for s in (1, 2, 3):
        now = [p for p in rows[s] if p >= 0]
        assert len(now) == len(held[s]) and rows[s][len(now):] == [-1] * (len(rows[s]) - len(now))
        seen += now
        for a, b in zip(held[s], now):
            assert torch.equal(k0[:, a].nan_to_num(nan=7.0), cache.k[:, b].nan_to_num(nan=7.0))
    assert sorted(seen) == list(range(live))


def test_compact_of_rows_wider_than_a_step(kv):
    # entries on both sides of every 1024th column, in rows whose lengths end before them
    n, pages = 3, 600
    cache = kv.PagedCache.create(1, pages, 8, 1, 16, n, 4100)
    at = [0, 1, 1022, 1023, 1024, 2047, 2048, 4000, 4095, 4096, 4099]
    used = list(range(1, pages, 2))
    table = torch.full((n, 4100), -1, dtype=torch.int32)
    for s in range(n):
        for i, c in enumerate(at):
            table[s, c] = used[(s * len(at) + i) * 7]
    cache.table.copy_(table)
    cache.refs[used] = 1
    m = ref.Model(cache)
    m.rows = table.tolist()
    m.compact()
    cache.compact()
    assert cache.table.tolist() == m.rows and cache.refs.tolist() == m.refs and cache.lens.tolist() == [0] * n
    cache.check()


@pytest.mark.parametrize("B", [3, 200])
def test_append_of_a_decreasing_cu_writes_no_place_but_the_sequences(kv, B):
    """cu [0, B, 2, 3, ...]: every token that is written lies at a place of one of the slots' last tokens; all else in
    the cache stays, and the status says so."""
    cache = ref.make_cache(kv, [40] * B, 16, 1, 64, BF, slots=B + 1)
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    cu[1] = B
    x = torch.randn(B, 2, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    k0, v0 = cache.k.clone(), cache.v.clone()
    cache.append(x, x[:, :1], x[:, 1:], cu)
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_LENGTH
    free = torch.ones(cache.k.shape[1:3], dtype=torch.bool, device="cuda")
    for b in range(B):  # the last tokens of a slot: as many as the call has rows, at most
        for p in range(max(0, 40 - B), 40):
            free[cache.table[b, p // 16].long(), p % 16] = False
    for x0, x1 in ((k0, cache.k), (v0, cache.v)):
        assert torch.equal(x0[0][free].nan_to_num(nan=7.0), x1[0][free].nan_to_num(nan=7.0))


@pytest.mark.parametrize("n", [257, 1500, 2500])
def test_long_lists_with_repeated_and_bad_slots(kv, n):
    """Above 256 entries grow marks slots in memory, above 1024 it takes the list part by part; free and fork look
    back over the whole list."""
    slots, rng = n // 2, random.Random(n)
    cache = kv.PagedCache.create(1, 4 * n, 8, 1, 16, slots, 12)
    m = ref.Model(cache)

    def some():
        return [rng.randrange(-2, slots + 2) if rng.random() < 0.2 else rng.randrange(slots) for _ in range(n)]

    for step in range(6):
        at, add = some(), [rng.choice([0, 1, 5, 9, 20]) for _ in range(n)]
        m.grow(at, add)
        cache.grow(vec(*at), vec(*add))
        m.same(cache, ("grow", step))
        src, dst = [rng.randrange(slots) for _ in range(n)], some()
        m.fork(src, dst)
        cache.fork(vec(*src), vec(*dst))
        m.same(cache, ("fork", step))
        at, keep = some(), [rng.choice([0, 3, 8, 17]) for _ in range(n)]
        m.free(at, keep)
        cache.free(vec(*at), vec(*keep))
        m.same(cache, ("free", step))
    assert m.bits & (kv.REPEATED | kv.BAD_SLOT) == kv.REPEATED | kv.BAD_SLOT
    everyone = list(range(slots)) * 2
    m.free(everyone)
    cache.free(vec(*everyone))
    m.same(cache, "all")
    assert m.refs.count(0) == len(m.refs)
