"""GPU parity of the paged-cache operators (include/fakv.h) with plain fp64 references, at the sizes, masks and
layouts where they can go wrong. Bounds are derived in _kv_ref.py."""
import math
import random

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


def vec(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def randn(*shape, dtype=F32, seed=0, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * mul).to(dtype).cuda()


SCALINGS = {"none": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=8.0),
            "bands": dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192),
            "yarn": dict(kind="yarn", factor=16.0, beta_fast=32.0, beta_slow=1.0, original=4096)}


# ---- rotary positions
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,HKV,D,rot,scaling", [
    (1, 4, 1, 128, 128, "none"), (37, 8, 2, 64, 32, "bands"), (5, 3, 3, 80, 40, "yarn"), (300, 5, 1, 96, 48, "ntk"),
    (3001, 2, 1, 128, 64, "linear"), (7, 1, 1, 16, 2, "none"), (64, 40, 8, 128, 126, "bands")])
def test_rope_and_its_gradient(kv, dtype, layout, T, H, HKV, D, rot, scaling):
    r = kv.Rope(D, rot, 500000.0, layout, SCALINGS[scaling])
    q, k = randn(T, H, D, dtype=dtype, seed=1), randn(T, HKV, D, dtype=dtype, seed=2)
    g = torch.Generator().manual_seed(3)
    for pos in (torch.randint(0, 1 << 20, (T,), generator=g), torch.randint(-5000, 5000, (T,), generator=g).int()):
        pos = pos.cuda()
        for inverse in (False, True):
            got = (r.backward if inverse else r.apply)(q, k, pos)
            for x, y, n in ((q, got[0], "q"), (k, got[1], "k")):
                want, bound = ref.rotate(x, pos, rot, 500000.0, SCALINGS[scaling], layout, inverse)
                ref.close(y, want, bound, (n, inverse))
                assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_gradient_against_differences(kv):
    # d/dx of sum(w * apply(x)) by central differences of the linear map: exact up to fp32 rounding
    r = kv.Rope(32, 16, layout="interleaved", scaling=SCALINGS["yarn"])
    T, H = 3, 2
    x, w, pos = randn(T, H, 32, seed=1), randn(T, H, 32, seed=2), torch.tensor([0, 77, 4001]).cuda()
    grad, _ = r.backward(w, None, pos)
    for t, h, c in ((0, 0, 0), (1, 1, 5), (2, 0, 15), (2, 1, 20)):
        e = torch.zeros_like(x)
        e[t, h, c] = 1.0
        up, dn = r.apply(x + e, None, pos)[0], r.apply(x - e, None, pos)[0]
        diff = ((up.double() - dn.double()) / 2 * w.double()).sum()
        # 2 x (32 values of size < 8, each to a few 2^-24)
        assert abs(diff - grad[t, h, c].double()) < 64 * 8 * 2.0 ** -22


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_in_place_strided_and_without_k(kv, dtype, layout):
    r = kv.Rope(64, 32, layout=layout)
    pos = torch.arange(1000, 1019).cuda()
    packed = randn(19, 6, 64, dtype=dtype, seed=4)  # 4 heads of q, then 2 of k, as one projection leaves them
    before = packed.clone()
    a, b = r.apply(packed[:, :4], packed[:, 4:], pos)
    assert torch.equal(packed, before)
    r.apply(packed[:, :4], packed[:, 4:], pos, out=(packed[:, :4], packed[:, 4:]))
    assert torch.equal(packed[:, :4], a) and torch.equal(packed[:, 4:], b)
    only, none = r.apply(before[:, :4], None, pos)
    assert none is None and torch.equal(only, a)
    # rows whose address or stride is not a multiple of 16 bytes
    wide = torch.zeros(19, 4 * 64 + 1, dtype=dtype, device="cuda")
    odd = wide[:, 1:].unflatten(1, (4, 64))
    odd.copy_(before[:, :4])
    assert torch.equal(r.apply(odd, None, pos)[0], a)
    assert r.apply(before[:0, :4], before[:0, 4:], pos[:0])[0].shape == (0, 4, 64)


# ---- append
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,lens,page,layout", [
    ([1], [1], 8, "tokens"), ([1, 1, 1], [5, 16, 17], 16, "tokens"), ([3, 0, 40, 1], [3, 9, 100, 33], 8, "heads"),
    ([1] * 70, [3 + i for i in range(70)], 32, "tokens"), ([700, 1], [700, 1024], 256, "heads")])
def test_append_writes_each_token_to_its_place(kv, dtype, new, lens, page, layout):
    B, H, HKV, D = len(new), 6, 2, 64
    order = torch.randperm(B + 2, generator=torch.Generator().manual_seed(1))[:B].tolist()
    cache = ref.make_cache(kv, lens, page, HKV, D, dtype, planes=2, slots=B + 2, order=order, layout=layout)
    k0, v0 = cache.k.clone(), cache.v.clone()
    T, pad = sum(new), 3
    q, k, v = (randn(T + pad, h, D, dtype=dtype, seed=i) for i, h in enumerate((H, HKV, HKV)))
    rope = kv.Rope(D, 32, layout="half", scaling=SCALINGS["linear"])
    out = torch.full_like(q, 9.0)
    slots = torch.tensor(order, dtype=torch.int32).cuda()
    assert cache.append(q, k, v, cu_of(new), slots, rope, layer=1, out=out) is out
    cache.check()
    assert bool((out[T:] == 9.0).all())
    pos = torch.cat([torch.arange(n - a, n) for a, n in zip(new, lens)] + [torch.zeros(0).long()]).cuda()
    want, bound = ref.rotate(q[:T], pos, 32, 10000.0, SCALINGS["linear"], "half")
    ref.close(out[:T], want, bound, "q")
    # k as rope.apply makes it, v as it is, in the second plane; everything else untouched
    rk = rope.apply(k[:T], None, pos)[0]
    at = 0
    for b, (a, n) in enumerate(zip(new, lens)):
        for i in range(a):
            p = n - a + i
            page_no, off = int(cache.table[order[b], p // page]), p % page
            for x, y in ((k0, rk), (v0, v)):
                if layout == "tokens":
                    x[1, page_no, off] = y[at + i]
                else:
                    x[1, page_no, :, off] = y[at + i]
        at += a
    assert torch.equal(cache.k.nan_to_num(nan=7.0), k0.nan_to_num(nan=7.0))
    assert torch.equal(cache.v.nan_to_num(nan=7.0), v0.nan_to_num(nan=7.0))
    # without positions, and without q
    cache.k.zero_()
    cache.append(None, k, v, cu_of(new), slots, layer=0)
    cache.check()
    if new[0]:
        p = lens[0] - new[0]
        x = cache.k[0, int(cache.table[order[0], p // page])]
        assert torch.equal(x[p % page] if layout == "tokens" else x[:, p % page], k[0])
    got = cache.append(q, k, v, cu_of(new), slots)
    assert torch.equal(got[:T], q[:T])


def test_append_in_place_one_token_and_one_head(kv):
    # contiguous in memory, whatever the strides of an extent of one say
    rope = kv.Rope(64)
    for H, HKV, T, make in ((4, 2, 1, lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)),
                            (1, 1, 5, lambda x: x.as_strided(x.shape, (64, 256, 1)))):
        cache = ref.make_cache(kv, [9], 8, HKV, 64, BF)
        q, k = randn(T, H, 64, dtype=BF, seed=1), randn(T, HKV, 64, dtype=BF, seed=2)
        want = cache.append(q, k, k, cu_of([T]), rope=rope)
        x = make(q.clone())
        assert x.is_contiguous() and cache.append(x, k, k, cu_of([T]), rope=rope, out=x) is x
        assert torch.equal(x, want)
        cache.check()


def test_append_leaves_out_what_the_table_refuses(kv):
    cache = ref.make_cache(kv, [20, 20, 20, 20], 16, 1, 16, BF, poison=False)
    before = cache.k.clone(), cache.v.clone()
    cache.table[0, 1] = 10 ** 6     # token 19 of slot 0: no page
    cache.lens[1] = -4              # no length
    cache.lens[2] = 0               # fewer tokens than new
    new = [1, 1, 1, 1]
    slots = torch.tensor([0, 1, 2, 77], dtype=torch.int32).cuda()
    x = randn(4, 1, 16, dtype=BF)
    cache.append(x, x, x, cu_of(new), slots)
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_PAGE | kv.BAD_LENGTH | kv.BAD_SLOT
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
    cache.check()  # read and cleared


# ---- attention
CASES = [
    # new, lens, H, HKV, D, page, causal, window
    ([1], [1], 1, 1, 16, 8, True, 0),
    ([1], [17], 4, 1, 128, 16, True, 0),
    ([1, 1, 1], [0, 5, 1000], 8, 2, 64, 16, True, 0),            # an empty sequence
    ([1] * 40, [7 * i + 1 for i in range(40)], 4, 2, 80, 8, True, 0),
    ([1], [40000], 16, 2, 128, 64, True, 0),                      # split over many CTAs
    ([3, 5, 0, 2], [300, 5, 9, 64], 6, 2, 96, 32, True, 0),       # drafts; rep 3; no new tokens
    ([4, 1], [513, 700], 4, 4, 64, 128, True, 100),               # windowed
    ([4, 2], [513, 300], 4, 2, 32, 1024, False, 0),               # not causal
    ([5, 7], [200, 7], 7, 1, 48, 16, False, 20),                  # window without causal
    ([3], [2], 2, 1, 64, 16, True, 0),                            # more new tokens than length: row 0 sees nothing
    ([33, 1, 129], [33, 500, 2000], 10, 2, 128, 16, True, 0),     # chunks
    ([200], [3000], 8, 1, 64, 8, True, 333),
    ([1, 300, 1, 17], [900, 300, 64, 1024], 4, 1, 112, 256, True, 0),
    ([65], [65], 64, 1, 64, 16, True, 0),                         # 64 heads on one kv head
    ([2], [300], 128, 1, 32, 16, True, 0),
    ([1] * 150, [(37 * i) % 211 for i in range(150)], 2, 1, 32, 16, True, 0),       # more sequences than a warp looks at
    ([1] * 40 + [700, 1, 0, 90], [50 + i for i in range(40)] + [800, 3, 40, 90], 4, 2, 64, 16, True, 0),
    ([0, 0, 700, 0, 300, 1], [10, 0, 700, 5, 1000, 999], 8, 2, 64, 32, True, 128),   # few sequences of many tiles
    ([1] * 3, [5000, 4999, 1], 4, 4, 128, 8, True, 0),
    ([8] * 5, [100, 2000, 8, 9, 700], 16, 8, 128, 16, True, 0),
    ([4] * 6, [1000, 40, 4, 600, 601, 2222], 32, 8, 80, 64, True, 50),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend(kv, dtype, case):
    new, lens, H, HKV, D, page, causal, window = CASES[case]
    B, pad = len(new), 2
    layout = "heads" if case % 2 else "tokens"
    order = torch.randperm(B + 1, generator=torch.Generator().manual_seed(case))[:B].tolist()
    cache = ref.make_cache(kv, lens, page, HKV, D, dtype, seed=case, slots=B + 1, order=order, layout=layout)
    T = sum(new)
    one_term = dtype == BF and (T + pad) * (H // HKV) > 16 * B  # many rows: the probabilities as one bf16 term
    q = randn(T + pad, H, D, dtype=dtype, seed=case, mul=1.5)
    q[T:] = float("nan")
    for odt in (dtype, F32 if dtype == BF else BF):
        o = torch.full((T + pad, H, D), 9.0, dtype=odt, device="cuda")
        lse = torch.full((T + pad, H), 9.0, device="cuda")
        slots = torch.tensor(order, dtype=torch.int32).cuda()
        cache.attend(q, cu_of(new), slots, 0.11, causal, window, out=o, lse=lse)
        cache.check()
        if case != 9:
            ro, rl, bo, bl = ref.attend(cache, q[:T], new, order, 0.11, causal, window, 0, layout,
                                        one_term=one_term)
        else:  # positions -1, 0, 1
            c2 = ref.make_cache(kv, lens, page, HKV, D, dtype, seed=case, slots=B + 1, order=order, layout=layout)
            ro, rl, bo, bl = ref.attend(c2, q[1:T], [2], order, 0.11, causal, window, 0, layout, one_term)
            z = lambda x, v: torch.cat([torch.full_like(x[:1], v), x])  # noqa: E731
            ro, rl, bo, bl = z(ro, 0.0), z(rl, -math.inf), z(bo, 0.0), z(bl, 0.0)
        ref.close(o[:T], ro, bo, "O")
        assert torch.equal(torch.isneginf(lse[:T]), torch.isneginf(rl))
        fin = torch.isfinite(rl)
        ref.close(lse[:T][fin], rl[fin], bl[fin], "LSE")
        assert bool((o[T:] == 9.0).all()) and bool((lse[T:] == 9.0).all())
        o2, l2 = cache.attend(q, cu_of(new), slots, 0.11, causal, window, out_dtype=odt)
        assert torch.equal(o2[:T], o[:T]) and torch.equal(l2[:T], lse[:T])  # the same on every run


def test_attend_strided_q_and_planes(kv):
    new, lens = [3, 1], [50, 333]
    cache = ref.make_cache(kv, lens, 16, 2, 64, BF, planes=3)
    packed = randn(4, 12, 64, dtype=BF, seed=5)  # q, k and v heads of one projection
    q = packed[:, :8]
    for plane in range(3):
        o, lse = cache.attend(q, cu_of(new), layer=plane)
        ro, rl, bo, bl = ref.attend(cache, q, new, [0, 1], 0.125, True, 0, plane, one_term=True)
        ref.close(o, ro, bo, "O")
        ref.close(lse, rl, bl, "LSE")


def test_attend_pages_shared_within_a_kv_pair_tensor(kv):
    # K and V as the halves of one tensor: page stride twice the page
    both = randn(1, 40, 2, 16, 2, 64, dtype=BF, seed=6)
    k, v = both[:, :, 0], both[:, :, 1]
    table = torch.arange(40, dtype=torch.int32).reshape(2, 20).cuda()
    cache = kv.PagedCache(k, v, table, torch.tensor([300, 111], dtype=torch.int32).cuda(),
                          torch.ones(40, dtype=torch.int32).cuda())
    q = randn(2, 4, 64, dtype=BF, seed=7)
    o, lse = cache.attend(q, cu_of([1, 1]))
    ro, rl, bo, bl = ref.attend(cache, q, [1, 1], [0, 1], 0.125, True, 0, one_term=True)
    ref.close(o, ro, bo, "O")


@pytest.mark.parametrize("n", [1, 40])
def test_attend_broadcast_q_and_a_table_within_a_wider_one(kv, n):
    cache = ref.make_cache(kv, [200, 333], 16, 2, 64, BF, seed=4, max_pages=30)
    wide = torch.full((2, 50), 1 << 20, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + 30] = cache.table[:, :30]
    other = kv.PagedCache(cache.k, cache.v, wide[:, 7:37], cache.lens, cache.refs)
    q = randn(2 * n, 1, 64, dtype=BF, seed=5).expand(2 * n, 8, 64)
    o, lse = other.attend(q, cu_of([n, n]))
    other.check()
    ro, rl, bo, bl = ref.attend(cache, q, [n, n], [0, 1], 0.125, True, 0, one_term=n > 1)
    ref.close(o, ro, bo, "O")
    other.fork(vec(1), vec(0))
    assert torch.equal(wide[0, 7:7 + 21], wide[1, 7:7 + 21]) and bool((wide[:, :7] == 1 << 20).all())
    assert bool((wide[:, 37:] == 1 << 20).all())


def test_attend_with_bad_pages_slots_and_lengths(kv):
    cache = ref.make_cache(kv, [100, 100, 100], 16, 1, 64, BF)
    q = randn(4, 4, 64, dtype=BF)
    good, _ = cache.attend(q[:1], cu_of([1]))
    cache.table[1, 2] = -1
    cache.table[1, 3] = 1 << 20
    cache.lens[2] = 1 << 30
    o, lse = cache.attend(q, cu_of([1, 1, 1, 1]), torch.tensor([0, 1, 2, -9], dtype=torch.int32).cuda())
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_PAGE | kv.BAD_LENGTH | kv.BAD_SLOT
    assert torch.equal(o[:1], good) and bool(torch.isfinite(o).all())
    assert bool((o[2:] == 0).all()) and bool(torch.isneginf(lse[2:]).all())


def test_far_offsets_pass_32_bits(kv):
    # a cache of more than 2^32 elements: the pages at its end are read and written
    pages, page, HKV, D = 70000, 64, 8, 128
    k = torch.empty(1, pages, page, HKV, D, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    table = torch.arange(pages - 5, pages, dtype=torch.int32, device="cuda")[None].contiguous()
    cache = kv.PagedCache(k, v, table, torch.tensor([300], dtype=torch.int32).cuda(),
                          torch.zeros(pages, dtype=torch.int32).cuda())
    assert k.numel() > 1 << 32
    x = [randn(300, h, D, dtype=BF, seed=h) for h in (16, 8)]
    y = randn(300, 8, D, dtype=BF, seed=3)
    cache.append(x[0], x[1], y, cu_of([300]))
    assert torch.equal(k[0, -5:].reshape(-1, HKV, D)[:300], x[1])
    for n in (1, 300):
        o, lse = cache.attend(x[0][300 - n:], cu_of([n]))
        ro, rl, bo, bl = ref.attend(cache, x[0][300 - n:], [n], [0], D ** -0.5, True, 0, one_term=True)
        ref.close(o, ro, bo, "O")
    cache.refs[-5:] = 1
    cache.compact()
    cache.check()
    assert cache.table[0].tolist() == [0, 1, 2, 3, 4]
    assert torch.equal(k[0, :5].reshape(-1, HKV, D)[:300], x[1])


def test_attend_the_most_sequences(kv):
    B, D = 16384, 16
    lens = [1 + (7 * b) % 5 for b in range(B)]
    cache = ref.make_cache(kv, lens, 8, 1, D, BF, poison=False)
    q = randn(B, 2, D, dtype=BF, seed=3)
    cu = cu_of([1] * B)
    o, lse = cache.attend(q, cu)
    cache.check()
    pick = list(range(0, B, 331)) + [B - 1]
    ro, rl, bo, bl = ref.attend(cache, q[pick], [1] * len(pick), pick, 0.25, True, 0)
    ref.close(o[pick], ro, bo, "O")
    ref.close(lse[pick], rl, bl, "LSE")
    one = cache.append(q, q[:, :1], q[:, 1:], cu)
    assert torch.equal(one, q)
    assert torch.equal(cache.k[0, cache.table[:, 0].long()[pick], [lens[b] - 1 for b in pick]], q[pick, :1])


def test_one_slot_for_several_sequences(kv):
    # drafts of one sequence scored from the same slot
    cache = ref.make_cache(kv, [77, 200], 16, 2, 64, BF)
    q = randn(6, 4, 64, dtype=BF)
    slots = vec(1, 0, 1)
    o, lse = cache.attend(q, cu_of([2, 2, 2]), slots)
    ro, rl, bo, bl = ref.attend(cache, q, [2, 2, 2], [1, 0, 1], 0.125, True, 0)
    ref.close(o, ro, bo, "O")


@pytest.mark.parametrize("B", [3, 200])
def test_a_cu_that_decreases_plans_no_work(kv, B):
    cache = ref.make_cache(kv, [40] * B, 16, 1, 64, BF, poison=False)
    q = randn(B, 2, 64, dtype=BF)
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    cu[1] = B
    o, lse = torch.full((B, 2, 64), 9.0, dtype=BF, device="cuda"), torch.full((B, 2), 9.0, device="cuda")
    cache.attend(q, cu, out=o, lse=lse)
    with pytest.raises(kv.CacheError):
        cache.check()
    assert bool((o == 9.0).all()) and bool((lse == 9.0).all())
    k = cache.k.clone()
    cache.append(q, q[:, :1], q[:, 1:], cu)  # (rows find the sequences that they find; no token leaves its row)
    assert cache.k.shape == k.shape and bool(torch.isfinite(cache.k.float()).all())


@pytest.mark.parametrize("B,n", [(4, 1), (2, 60)])
def test_two_graphs_replayed_at_once(kv, B, n):
    caches = [ref.make_cache(kv, [9000 - i] * B, 16, 2, 64, BF, seed=i) for i in range(2)]
    q, cu = randn(B * n, 8, 64, dtype=BF), cu_of([n] * B)
    want = [c.attend(q, cu) for c in caches]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for c, s in zip(caches, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(c.attend(q, cu))
        graphs.append(g)
    for _ in range(20):
        for o in outs:
            o[0].fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


# ---- pages


@pytest.mark.parametrize("dtype,layout,max_pages", [(BF, "tokens", 9), (F32, "heads", 9), (BF, "tokens", 9000)])
def test_pages_random_walk_against_the_model(kv, dtype, layout, max_pages):
    rng = random.Random(11)
    cache = ref.make_cache(kv, [0, 5, 16, 33, 0, 8, 1, 0], 8, 2, 16, dtype, planes=2, extra=20, layout=layout,
                           max_pages=max_pages)
    m = ref.Model(cache)
    for step in range(120):
        n = rng.randrange(1, 7)
        slots = [rng.randrange(-1, 9) if rng.random() < 0.1 else rng.randrange(8) for _ in range(n)]
        op = rng.choice(["grow", "grow", "fork", "free", "compact"])
        if op == "grow":
            add = [rng.choice([0, 1, 3, 8, 20, -1 if rng.random() < 0.2 else 2]) for _ in slots]
            m.grow(slots, add)
            cache.grow(vec(*slots), vec(*add))
        elif op == "fork":
            src = [rng.randrange(8) for _ in slots]
            m.fork(src, slots)
            cache.fork(vec(*src), vec(*slots))
        elif op == "free":
            keep = None if rng.random() < 0.3 else [rng.choice([0, 1, 7, 8, 9, 40]) for _ in slots]
            m.free(slots, keep)
            cache.free(vec(*slots), None if keep is None else vec(*keep))
        else:
            m.compact()
            cache.compact()
        m.same(cache, (step, op, slots))


def test_grow_long_lists_and_long_entries(kv):
    # more entries than a planning block has threads, some needing many pages; then more than are free
    n = 2500
    cache = kv.PagedCache.create(1, 9000, 8, 1, 16, n, 40)
    m = ref.Model(cache)
    order = list(range(n))
    random.Random(3).shuffle(order)
    for seed in range(4):
        rng = random.Random(seed)
        add = [rng.choice([1, 2, 9, 30, 0]) for _ in order]
        m.grow(order, add)
        cache.grow(vec(*order), vec(*add))
        m.same(cache, seed)
    assert m.bits & 1  # (the last rounds asked for too much)


@pytest.mark.parametrize("pages,shift", [(4095, 0), (4097, 0), (20480, 0), (20483, 1), (70001, 3)])
def test_grow_finds_the_free_pages_of_a_mostly_full_pool(kv, pages, shift):
    # one free page in two hundred, none among the first 4096 but two, and counts at any address
    g = torch.Generator().manual_seed(pages)
    used = (torch.rand(pages, generator=g) >= 0.005).int()
    used[:4096] = 1
    used[[7, 4094]] = 0
    used[-1] = 0
    whole = torch.ones(pages + shift, dtype=torch.int32, device="cuda")
    refs = whole[shift:]
    refs.copy_(used)
    k = torch.zeros(1, pages, 8, 1, 16, device="cuda")
    n = 1500
    cache = kv.PagedCache(k, k.clone(), torch.full((n, 40), -1, dtype=torch.int32, device="cuda"),
                          torch.zeros(n, dtype=torch.int32, device="cuda"), refs)
    m = ref.Model(cache)
    for slots, add in (((0, 1), (8, 17)), (range(2, 40), [9] * 38), (range(n), [1] * n)):
        m.grow(list(slots), list(add))
        cache.grow(vec(*slots), vec(*add))
        m.same(cache, (pages, len(add)))


def test_grow_refuses_more_than_any_row_or_sum_holds(kv):
    cache = kv.PagedCache.create(1, 64, 8, 1, 16, 3, 1 << 27)
    cache.grow(vec(0, 1, 2), vec((1 << 30) - 8, 1 << 30, 16))
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.NO_PAGES and cache.lens.tolist() == [0, 0, 0] and int(cache.refs.sum()) == 0


def test_fork_exchanges_slots(kv):
    cache = ref.make_cache(kv, [20, 9, 30], 8, 1, 16, BF)
    m = ref.Model(cache)
    rows = [list(r) for r in m.rows]
    m.fork([0, 1, 2], [1, 2, 0])
    cache.fork(vec(0, 1, 2), vec(1, 2, 0))
    m.same(cache, "rotation")
    assert m.rows[1] == rows[0] and m.refs.count(1) == sum(map(len, rows))


@pytest.mark.parametrize("n,max_pages", [(32, 256), (33, 256), (32, 257), (1, 256), (200, 40)])
def test_fork_of_lists_and_rows_of_any_size(kv, n, max_pages):
    # full, empty and half rows; permuted, so that every slot is a source and a destination
    cache = kv.PagedCache.create(1, n * max_pages + 4, 8, 1, 16, n + 1, max_pages)
    m = ref.Model(cache)
    order, add = list(range(n)), [(i % 3) * 4 * max_pages for i in range(n)]
    add[0] = 8 * max_pages
    m.grow(order, add)
    cache.grow(vec(*order), vec(*add))
    src = [(5 * i + 3) % n for i in range(n)] if n % 5 else order
    for dst in (order, [n] + order[1:], order[::-1]):
        m.fork(src, dst)
        cache.fork(vec(*src), vec(*dst))
        m.same(cache, dst[:2])


def test_compact_of_full_empty_and_large_caches(kv):
    for pages, gone in ((1, 0.0), (37, 1.0), (64, 0.0), (9001, 0.4), (65536, 0.5), (70001, 0.3)):
        g = torch.Generator().manual_seed(pages)
        used = (torch.rand(pages, generator=g) >= gone).int()
        k = torch.arange(pages * 8 * 16, device="cuda").float().reshape(1, pages, 8, 1, 16)
        live = torch.nonzero(used)[:, 0].int()
        live = live[torch.randperm(len(live), generator=g)]
        table = torch.full((2, pages + 1), -1, dtype=torch.int32)
        table[1, :len(live)] = live
        cache = kv.PagedCache(k, k.clone(), table.cuda(), vec(0, 8 * len(live)), used.cuda())
        m = ref.Model(cache)
        m.compact()
        cache.compact()
        m.same(cache, pages)


# ---- together
def plain_step(c, k_all, v_all, q, scale):
    """Attention of q [n, H, D] (the last n positions) over k_all, v_all [len, HKV, D], fp64."""
    group = q.shape[1] // k_all.shape[1]
    k, v = (x.repeat_interleave(group, 1).double() for x in (k_all, v_all))
    z = torch.einsum("thd,jhd->htj", q.double(), k) * scale
    n, size = q.shape[0], k.shape[0]
    hide = torch.arange(size, device=q.device)[None] > torch.arange(size - n, size, device=q.device)[:, None]
    return torch.einsum("htj,jhd->thd", z.masked_fill(hide, -math.inf).softmax(-1), v)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_fork_decode_free_compact(kv, dtype):
    """A prompt in two chunks, two samples forked from it, decoding by graph replay, one sample leaving, compaction:
    every output against attention over the tokens as they were given."""
    L, H, HKV, D, page = 2, 4, 2, 64, 16
    cache = kv.PagedCache.create(L, 40, page, HKV, D, 4, 8, dtype)
    rope = kv.Rope(D, scaling=SCALINGS["bands"], base=500000.0)
    seen = {s: [([], []) for _ in range(L)] for s in range(3)}  # what each slot should hold
    seed = [100]

    def tokens(n):
        seed[0] += 1
        return [randn(n, h, D, dtype=dtype, seed=seed[0] * 10 + i) for i, h in enumerate((H, HKV, HKV))]

    def note(slot, layer, k, v, start):
        pos = torch.arange(start, start + k.shape[0]).cuda()
        seen[slot][layer][0].append(rope.apply(k, None, pos)[0])
        seen[slot][layer][1].append(v)

    def check(slot, layer, q, o):
        k, v = (torch.cat(x) for x in seen[slot][layer])
        pos = torch.arange(k.shape[0] - q.shape[0], k.shape[0]).cuda()
        want = plain_step(None, k, v, rope.apply(q, None, pos)[0], D ** -0.5)
        # the bounds of _kv_ref.attend at these sizes: |v| < 5, e below 2e-4, P to 2^-8 (bf16) or 2^-21
        lim = 5 * (2 * 2e-4 + 2.0 ** -8) if dtype == BF else 5 * 2 * 2e-4
        ref.close(o, want, torch.full_like(want, lim), (slot, layer))

    start = 0
    for n in (37, 12):
        cache.grow(vec(0), vec(n))
        for layer in range(L):
            q, k, v = tokens(n)
            qr = cache.append(q, k, v, cu_of([n]), vec(0), rope, layer)
            o, _ = cache.attend(qr, cu_of([n]), vec(0), layer=layer)
            note(0, layer, k, v, start)
            check(0, layer, q, o)
        start += n
    cache.fork(vec(0, 0), vec(1, 2))
    for s in (1, 2):
        seen[s] = [(list(k), list(v)) for k, v in seen[0]]
    slots, ones, cu = vec(0, 1, 2), vec(1, 1, 1), cu_of([1, 1, 1])
    buf = [tokens(3) for _ in range(L)]
    outs = [torch.empty(3, H, D, dtype=dtype, device="cuda") for _ in range(L)]

    def step():
        cache.grow(slots, ones)
        for layer in range(L):
            q = cache.append(*buf[layer], cu, slots, rope, layer)
            cache.attend(q, cu, slots, layer=layer, out=outs[layer])

    graph = None
    for i in range(20):
        for layer in range(L):
            for x, y in zip(buf[layer], tokens(3)):
                x.copy_(y)
        if i == 2:
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        for layer in range(L):
            q, k, v = buf[layer]
            for s in range(3):
                note(s, layer, k[s:s + 1].clone(), v[s:s + 1].clone(), start)
                check(s, layer, q[s:s + 1], outs[layer][s:s + 1])
        start += 1
    cache.check()
    before = int((cache.refs > 0).sum())
    cache.free(vec(0))
    cache.compact()
    live = int((cache.refs > 0).sum())
    assert live < before and bool((cache.refs[:live] > 0).all())
    seen[0] = [([], []) for _ in range(L)]
    cache.grow(vec(1, 2), vec(2, 2))
    cu2 = cu_of([2, 2])
    for layer in range(L):
        q, k, v = tokens(4)
        qr = cache.append(q, k, v, cu2, vec(1, 2), rope, layer)
        o, _ = cache.attend(qr, cu2, vec(1, 2), layer=layer)
        for i, s in enumerate((1, 2)):
            note(s, layer, k[2 * i:2 * i + 2], v[2 * i:2 * i + 2], start)
            check(s, layer, q[2 * i:2 * i + 2], o[2 * i:2 * i + 2])
    cache.check()


def test_calls_on_a_stream_of_their_own(kv):
    cache = ref.make_cache(kv, [100, 2000], 16, 2, 64, BF)
    q = randn(2, 8, 64, dtype=BF)
    want = cache.attend(q, cu_of([1, 1]))
    s = torch.cuda.Stream()
    cu = cu_of([1, 1])
    torch.cuda.synchronize()
    got = [cache.attend(q, cu, stream=s) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(s)
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_streams_at_once_do_not_share_scratch(kv):
    a = ref.make_cache(kv, [30000], 16, 2, 128, BF, seed=1)
    b = ref.make_cache(kv, [29000], 16, 2, 128, BF, seed=2)
    q, cu = randn(1, 8, 128, dtype=BF), cu_of([1])
    want = [c.attend(q, cu) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, c in enumerate((a, b)):
            got[i].append(c.attend(q, cu, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_no_sequences_and_no_rows(kv):
    cache = ref.make_cache(kv, [10], 16, 1, 64, BF)
    q = randn(3, 2, 64, dtype=BF)
    o, lse = cache.attend(q, cu_of([]))
    assert o.shape == (3, 2, 64)
    o = torch.full((3, 2, 64), 9.0, dtype=BF, device="cuda")
    l = torch.full((3, 2), 9.0, device="cuda")
    cache.attend(q, cu_of([0]), out=o, lse=l)       # a sequence without new tokens
    assert bool((o == 9.0).all()) and bool((l == 9.0).all())
    cache.attend(q[:0], cu_of([0]))
    cache.append(q[:0], q[:0, :1], q[:0, :1], cu_of([0]))
    cache.grow(vec(), vec())
    cache.fork(vec(), vec())
    cache.free(vec())
    cache.check()
