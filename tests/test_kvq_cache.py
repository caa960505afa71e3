"""GPU tests of the cache in 4 or 8 bits as it is used: its pages, steps captured into graphs, streams, values that are
no numbers, rows of others, long caches; and a run of its calls together."""
import math

import pytest
import torch

import _kv_ref
import _kvq_ref as ref
from test_kvq_gpu import BF, F32, cu_of, randn, vec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_fa_fwd_02_gb300 import kv as m
    return m


@pytest.mark.parametrize("D,bits,group,page,planes", [(128, 4, 64, 8, 2), (96, 8, 96, 32, 1), (48, 4, 48, 16, 3), (16, 8, 16, 8, 1)])
def test_page_calls_do_what_they_do_to_a_plain_cache(kv, D, bits, group, page, planes):
    """grow, fork, free and compact on both kinds of cache, the same tables; every token keeps what it holds."""
    lens, HKV, slots, width = [3 * page + 5, page, 2 * page - 1, 7], 2, 9, 12
    q, _ = ref.make(kv, lens, page, HKV, D, bits, group, BF, planes=planes, slots=slots, extra=40, max_pages=width, seed=4)
    p = kv.PagedCache.create(planes, q.k.shape[1], page, HKV, 16, slots, width)
    for x in ("table", "lens", "refs"):
        getattr(p, x).copy_(getattr(q, x))
    before = [[ref.held(q, s, l)[i][0] for s in range(4) for i in range(2)] for l in range(planes)]

    def both(what, *a):
        for c in (q, p):
            getattr(c, what)(*a)
            c.check()
        for x in ("table", "lens", "refs"):
            assert torch.equal(getattr(q, x), getattr(p, x)), (what, x)

    def tokens_are(slot, of, n):
        for l in range(planes):
            for i in range(2):
                assert torch.equal(ref.held(q, slot, l)[i][0][:n], before[l][2 * of + i][:n])

    both("fork", vec(0, 2, 0), vec(4, 5, 6))
    both("grow", vec(4, 5, 6, 1), vec(1, page, 3, 2))  # shared last pages are copied first
    for slot, of in ((4, 0), (5, 2), (6, 0), (0, 0), (1, 1)):
        tokens_are(slot, of, lens[of])
    both("free", vec(0, 3), vec(page + 1, 0))
    both("free", vec(2))
    both("compact")
    for slot, of, n in ((4, 0, lens[0]), (5, 2, lens[2]), (6, 0, lens[0]), (0, 0, page + 1), (1, 1, lens[1])):
        tokens_are(slot, of, n)
    for c in (q, p):
        c.grow(vec(8, 8, 99), vec(1, 1, 1))
        with pytest.raises(kv.CacheError) as e:
            c.check()
        assert e.value.bits == kv.REPEATED | kv.BAD_SLOT


@pytest.mark.parametrize("bits,group", [(4, 64), (8, 128)])
def test_a_models_steps_together(kv, bits, group):
    """Two layers, three sequences: a prompt's chunk, decoding steps, a fork, drafts and their rejection, all against fp64
    over what the cache holds, which is within half a step of what was given."""
    H, HKV, D, page, layers = 8, 2, 128, 16, 2
    cache = kv.QuantCache.create(layers, 60, page, HKV, D, 4, 24, bits, group)
    rope = kv.Rope(D, scaling=dict(kind="linear", factor=2.0))
    given = {}  # slot -> layer -> list of (rotated k, v)
    g = torch.Generator().manual_seed(7)

    def step(slots, new):
        cache.grow(vec(*slots), vec(*new))
        cu, T = cu_of(new), sum(new)
        for layer in range(layers):
            q, k, v = ((torch.randn(T, h, D, generator=g) * 1.5).to(BF).cuda() for h in (H, HKV, HKV))
            turned = cache.append(q, k, v, cu, vec(*slots), rope, layer)
            o, lse = cache.attend(turned, cu, vec(*slots), layer=layer)
            cache.check()
            many = T * (H // HKV) > 16 * len(slots)
            want, want_l, bo, bl = ref.attend(cache, turned, new, slots, D ** -0.5, True, 0, layer, many, False)
            _kv_ref.close(o.cpu(), want, bo, "O")
            assert bool(((lse.cpu().double() - want_l).abs() <= bl).all())
            at = 0
            for s, n in zip(slots, new):
                length = int(cache.lens[s])
                pos = torch.arange(length - n, length).cuda()
                x, e = _kv_ref.rotate(k[at:at + n], pos, D, 10000.0, dict(kind="linear", factor=2.0), "half")
                given.setdefault((s, layer), []).append((x.cpu(), e.cpu(), v[at:at + n].double().cpu()))
                at += n

    step([0, 1], [70, 33])
    for _ in range(3):
        step([1, 0], [1, 1])
    cache.fork(vec(0), vec(2))
    for layer in range(layers):
        given[2, layer] = list(given[0, layer])
    step([2, 1], [4, 1])
    cache.free(vec(2), torch.tensor([75], dtype=torch.int32).cuda())  # two of the four drafts stay
    cache.check()
    step([2, 0, 1], [1, 2, 40])
    assert cache.lens.tolist() == [75, 77, 76, 0]
    for (slot, layer), parts in given.items():
        if slot == 2:
            parts[-2] = tuple(x[:2] for x in parts[-2])
        k, v = cache.read(cu_of([int(cache.lens[slot])]), int(cache.lens[slot]), vec(slot), layer=layer, out_dtype=F32)
        (hk, sk, _, _), (hv, sv, _, _) = ref.held(cache, slot, layer)
        assert torch.equal(k.cpu(), hk.float()) and torch.equal(v.cpu(), hv.float())
        want_k, e, want_v = (torch.cat(x) for x in zip(*parts))
        half = 0.5 + 255 * 3 * 2.0 ** -24
        assert bool(((hk - want_k).abs() <= sk * half + e).all()) and bool(((hv - want_v).abs() <= sv * half).all())


def test_read_feeds_the_contiguous_attention(kv):
    """K and V of a prefix, read back, through fa.forward: the same as attending over the cache."""
    from attention_fa_fwd_02_gb300 import fa
    n, H, HKV, D = 300, 8, 2, 128
    cache, _ = ref.make(kv, [n], 16, HKV, D, 8, 128, BF)
    q = randn(n, H, D, dtype=BF, seed=3)
    k, v = cache.read(cu_of([n]), n)
    o, _ = fa.forward(*(x.transpose(0, 1).contiguous()[None] for x in (q, k, v)), causal=True)
    p, _ = cache.attend(q, cu_of([n]), out_dtype=F32)
    # the values rounded to bf16 (2^-9 at most), fp16 in the tiles (2^-11); the forward's own P (2^-11): an O is an average
    # of values of that size, and scores of size up to 10 move by 10 * 2^-9
    assert float((o[0].transpose(0, 1) - p).norm() / p.norm()) < 0.03


def test_captured_steps_replay_as_lengths_move(kv):
    H, HKV, D, B = 8, 2, 128, 3
    out = []
    for captured in (False, True):
        cache, _ = ref.make(kv, [40, 7, 100], 16, HKV, D, 4, 64, BF, extra=30, max_pages=12, seed=5)
        rope = kv.Rope(D)
        q, k, v = randn(B, H, D, dtype=BF, seed=1), randn(B, HKV, D, dtype=BF, seed=2), randn(B, HKV, D, dtype=BF, seed=3)
        slots, one, cu = vec(0, 1, 2), vec(1, 1, 1), cu_of([1, 1, 1])
        wide, cu_w = randn(B * 40, H, D, dtype=BF, seed=4), cu_of([40, 7, 40])

        def step():
            cache.grow(slots, one)
            t = cache.append(q, k, v, cu, slots, rope)
            a = cache.attend(t, cu, slots)
            b = cache.attend(wide, cu_w, slots)  # rows past cu[-1] are not written
            c = cache.read(cu, B, slots)
            return *a, b[0][:87], b[1][:87], *c

        if captured:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                step()
            torch.cuda.synchronize()
            cache, _ = ref.make(kv, [40, 7, 100], 16, HKV, D, 4, 64, BF, extra=30, max_pages=12, seed=5)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                r = step()
            got = []
            for _ in range(12):
                g.replay()
                got.append([x.clone() for x in r])
        else:
            got = [[x.clone() for x in step()] for _ in range(12)]
        cache.check()
        out.append(got)
    for a, b in zip(*out):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_and_two_streams_share_nothing(kv):
    H, HKV, D = 8, 2, 64
    caches = [ref.make(kv, [500 + 100 * i, 33], 16, HKV, D, 8, 64, BF, seed=i)[0] for i in range(2)]
    qs = [randn(50, H, D, dtype=BF, seed=10 + i) for i in range(2)]
    cus = [cu_of([40, 10]), cu_of([1, 1])]
    want = [[c.attend(q[:n], cu) for cu, n in zip(cus, (50, 2))] for c, q in zip(caches, qs)]
    graphs, res = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append([caches[i].attend(qs[i][:n], cu) for cu, n in zip(cus, (50, 2))])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, res):
        for (o, l), (p, m) in zip(a, b):
            assert torch.equal(o, p) and torch.equal(l, m)
    # a call on a stream of its own
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, l = caches[0].attend(qs[0], cus[0], stream=s)
    k, v = caches[0].read(cus[1], 2, stream=s)
    s.synchronize()
    assert torch.equal(o, want[0][0][0]) and torch.equal(l, want[0][0][1])
    assert torch.equal(k, caches[0].read(cus[1], 2)[0])


@pytest.mark.parametrize("dtype,rows", [(BF, 4), (F32, 4), (BF, 40)])
@pytest.mark.parametrize("bits", [4, 8])
def test_values_that_are_no_numbers_stay_with_who_sees_them(kv, dtype, rows, bits):
    """A token whose k or v holds NaN or infinity: rows that see it are NaN, rows before it are as if it held zeros."""
    D, H, HKV, old = 64, 4, 1, 90
    clean, given = ref.make(kv, [old + rows], 16, HKV, D, bits, D, dtype, seed=6, planes=4)
    q, cu = randn(rows, H, D, dtype=dtype, seed=1), cu_of([rows])
    bad = rows // 2  # of the new tokens
    for layer, (which, value) in enumerate((("k", math.nan), ("v", math.inf), ("v", -math.nan), ("k", -math.inf))):
        o, l = clean.attend(q, cu, layer=layer)
        k, v = (x.clone() for x in given[layer])
        (k if which == "k" else v)[old + bad, 0, 5] = value
        clean.append(None, k, v, cu_of([old + rows]), layer=layer)
        p, m = clean.attend(q, cu, layer=layer)
        clean.check()
        assert torch.equal(p[:bad], o[:bad]) and torch.equal(m[:bad], l[:bad])
        assert bool(torch.isnan(p[bad:]).any(-1).all())
        assert not bool(torch.isnan(o).any())


@pytest.mark.parametrize("dtype,rows", [(BF, 3), (F32, 3), (BF, 60)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_no_number_in_a_row_of_q_stays_in_it(kv, dtype, rows, value):
    cache, _ = ref.make(kv, [400], 16, 1, 128, 4, 64, dtype)
    q, cu = randn(rows, 4, 128, dtype=dtype, seed=2), cu_of([rows])
    for odt in (BF, F32):
        o, l = cache.attend(q, cu, out_dtype=odt)
        r = q.clone()
        r[1, 2, 77] = value
        p, m = cache.attend(r, cu, out_dtype=odt)
        cache.check()
        assert bool(torch.isnan(p[1, 2]).all()) and bool(torch.isnan(m[1, 2]))
        p[1, 2], m[1, 2] = o[1, 2], l[1, 2]
        assert torch.equal(p, o) and torch.equal(m, l)


@pytest.mark.parametrize("dtype,rows", [(BF, 2), (F32, 4), (BF, 50)])
def test_no_bit_depends_on_rows_of_others(kv, dtype, rows):
    cache, _ = ref.make(kv, [700], 16, 2, 128, 8, 128, dtype)
    q, cu = randn(rows, 8, 128, dtype=dtype, seed=2), cu_of([rows])
    o, l = cache.attend(q, cu)
    r = q.clone()
    r[:, ::2] *= 30  # half of the heads' scores are others, and their maxima move at other keys
    p, m = cache.attend(r, cu)
    assert torch.equal(p[:, 1::2], o[:, 1::2]) and torch.equal(m[:, 1::2], l[:, 1::2])


@pytest.mark.parametrize("rows", [1, 40])
def test_sizes_of_values_far_from_one(kv, rows):
    """K of 1e-20 with q of 1e20, V of 1e25, V of 1e-25; V that grows by 2^40 on the way, and K beside zeros."""
    D, n = 64, 600
    for bits in (4, 8):
        cache, given = ref.make(kv, [n], 16, 1, D, bits, D, BF, planes=1)
        k, v = given[0]
        q, cu = randn(rows, 2, D, dtype=BF, seed=5), cu_of([rows])
        for fk, fq, fv in ((1e-20, 1e20, 1e25), (1e15, 1e-15, 1e-25), (0.0, 1.0, 1.0), (1.0, 0.0, 1.0)):
            cache.append(None, k * fk, v * fv, cu_of([n]))
            o, l = cache.attend(q * fq, cu)
            want, want_l, bo, bl = ref.attend(cache, q * fq, [rows], [0], D ** -0.5, True, 0, 0, rows > 8)
            _kv_ref.close(o.cpu(), want, bo, (fk, fq, fv))
            assert bool(((l.cpu().double() - want_l).abs() <= bl).all())
        steps = torch.ones(n, 1, 1, device="cuda")
        steps[200:] = 2.0 ** 20
        steps[400:] = 2.0 ** 40
        cache.append(None, k, v * steps.to(BF), cu_of([n]))
        o, l = cache.attend(q, cu)
        want, _, bo, _ = ref.attend(cache, q, [rows], [0], D ** -0.5, True, 0, 0, rows > 8)
        _kv_ref.close(o.cpu(), want, bo, "steps")


def test_missing_pages_read_as_zeros(kv):
    for rows in (1, 30):
        cache, _ = ref.make(kv, [200], 16, 2, 64, 4, 64, BF)
        zero = ref.make(kv, [200], 16, 2, 64, 4, 64, BF)[0]
        p = int(cache.table[0, 5])
        for x in (zero.k, zero.v):
            x[0, p] = 0
        q, cu = randn(rows, 4, 64, dtype=BF, seed=1), cu_of([rows])
        want = zero.attend(q, cu)
        for entry in (-1, 1 << 20):
            cache.table[0, 5] = entry
            got = cache.attend(q, cu)
            with pytest.raises(kv.CacheError) as e:
                cache.check()
            assert e.value.bits == kv.BAD_PAGE
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_slots_lengths_and_cu(kv):
    cache, _ = ref.make(kv, [50, 60], 16, 1, 64, 8, 64, BF, slots=3)
    q, cu = randn(6, 2, 64, dtype=BF), cu_of([2, 2, 2])
    cache.lens[2] = 100000
    o, l = cache.attend(q, cu, vec(0, 7, 2))
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_SLOT | kv.BAD_LENGTH
    assert bool((o[2:] == 0).all()) and bool((l[2:] == -math.inf).all()) and bool(torch.isfinite(l[:2]).all())
    k0 = cache.k.clone()
    x = randn(6, 1, 64, dtype=BF)
    cache.append(None, x, x, cu, vec(9, 2, -1))
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_SLOT | kv.BAD_LENGTH and torch.equal(cache.k, k0)
    down = torch.tensor([0, 4, 2], dtype=torch.int32).cuda()
    out = torch.full_like(q, 3.0)
    cache.attend(q, down, vec(0, 1), out=out)
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_LENGTH and bool((out == 3.0).all())  # nothing is done with one that decreases
    cache.append(None, x, x, down, vec(0, 1))
    cache.read(down, 6, vec(0, 1))
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_LENGTH


@pytest.mark.parametrize("new", [1, 24, 40])
def test_offsets_past_32_bits(kv, new):
    """A plane whose pages lie up to 9 GB from its beginning."""
    page, HKV, D, pages = 64, 4, 128, 256000
    k = torch.empty(1, pages, HKV, kv.QuantCache.block_bytes(page, D, 8, 128), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    n = 5 * page + 9
    table = torch.full((1, 8), -1, dtype=torch.int32)
    table[0, :6] = torch.tensor([0, pages - 1, 130000, 65001, 200000, pages - 2], dtype=torch.int32)
    cache = kv.QuantCache(k, v, table.cuda(), vec(n), torch.zeros(pages, dtype=torch.int32, device="cuda"), page, D, 8, 128)
    given = [randn(n, HKV, D, dtype=BF, seed=i) for i in range(2)]
    cache.append(None, *given, cu_of([n]))
    small = kv.QuantCache.create(1, 8, page, HKV, D, 1, 8, 8, 128)
    small.table[0, :6] = torch.arange(6, dtype=torch.int32)
    small.lens.fill_(n)
    small.append(None, *given, cu_of([n]))
    q = randn(new, 8, D, dtype=BF, seed=9)
    for a, b in zip(cache.attend(q, cu_of([new])), small.attend(q, cu_of([new]))):
        assert torch.equal(a, b)
    for a, b in zip(cache.read(cu_of([n]), n), small.read(cu_of([n]), n)):
        assert torch.equal(a, b)
    cache.check()


def test_thousands_of_sequences(kv):
    """More sequences than a warp plans by itself, most of them empty; a table within a wider one; pages spaced apart."""
    B, HKV, D, page = 5000, 1, 32, 8
    lens = [(i * 7) % 23 if i % 3 == 0 else 0 for i in range(B)]
    cache, _ = ref.make(kv, lens, page, HKV, D, 4, D, BF, max_pages=4)
    wide = torch.full((B, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:6] = cache.table
    big = [torch.empty(1, cache.k.shape[1], HKV, 2, cache.k.shape[3], dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y in zip(big, (cache.k, cache.v)):
        x[:, :, :, 0] = y
    apart = kv.QuantCache(big[0][:, :, :, 0], big[1][:, :, :, 0], wide[:, 2:6], cache.lens, cache.refs, page, D, 4)
    new = [1 if n else 0 for n in lens]
    q = randn(sum(new), 2, D, dtype=BF)
    a, b = cache.attend(q, cu_of(new)), apart.attend(q, cu_of(new))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    some = [i for i, n in enumerate(new) if n][::97]
    rows = [sum(new[:i]) for i in some]
    want, want_l, bo, bl = ref.attend(cache, q[rows], [1] * len(some), some, D ** -0.5, True, 0)
    _kv_ref.close(a[0][rows].cpu(), want, bo, "O")
    got = apart.read(cu_of(lens), sum(lens))
    for x, y in zip(got, cache.read(cu_of(lens), sum(lens))):
        assert torch.equal(x, y)
    cache.check()
    apart.check()


@pytest.mark.parametrize("bits", [4, 8])
def test_thousands_of_sequences_chunks(kv, bits):
    """More sequences than the tile kernel has threads, each with new tokens of its own."""
    B, D, page = 1500, 16, 8
    lens = [(i * 7) % 41 if i % 3 else 90 for i in range(B)]
    new = [n if i % 3 else 70 for i, n in enumerate(lens)]
    cache, _ = ref.make(kv, lens, page, 1, D, bits, D, BF)
    T = sum(new)
    q = randn(T, 2, D, dtype=BF, mul=1.5)
    assert T * 2 > 48 * B
    o, lse = cache.attend(q, cu_of(new))
    cache.check()
    for i in (0, 1, 2, 640, 1001, 1498, 1499):
        a = sum(new[:i])
        want, want_l, bo, bl = ref.attend(cache, q[a:a + new[i]], [new[i]], [i], D ** -0.5, True, 0, 0, True)
        _kv_ref.close(o[a:a + new[i]].cpu(), want, bo, i)
        assert bool(((lse[a:a + new[i]].cpu().double() - want_l).abs() <= bl).all())
