"""GPU parity of the cache in 4 or 8 bits (include/fakv.h) with its definition: codes and parameters bit for bit,
attention within bounds derived in _kvq_ref.py, at the sizes, masks and layouts where they can go wrong."""
import math

import pytest
import torch

import _kv_ref
import _kvq_ref as ref

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


def same(a, b):
    return torch.equal(a.nan_to_num(nan=12345.0), b.nan_to_num(nan=12345.0))


# ---- append
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,bits,group", ref.SHAPES)
def test_append_holds_the_definition_bit_for_bit(kv, dtype, D, bits, group):
    lens, new, page, HKV, planes = [21, 8, 1, 40], [21, 3, 1, 17], 8, 3, 2
    order = [4, 0, 2, 1]
    cache, _ = ref.make(kv, lens, page, HKV, D, bits, group, dtype, planes=planes, slots=5, order=order, stored=False)
    k0, v0 = cache.k.clone(), cache.v.clone()
    T, pad = sum(new), 2
    q, k, v = (randn(T + pad, h, D, dtype=dtype, seed=i) for i, h in enumerate((6, HKV, HKV)))
    # constants, one large column, denormals, the largest that has a scale; and what has none
    k[1], k[2, 0], k[3] = 0.75, k[2, 0] * 1e-39, -0.0
    k[4, :, 3], v[5, :, 1] = 300.0, -(2.0 ** 125)
    k[6, 1, 2], v[7, 0, 0], v[8, 2, 5] = math.nan, math.inf, 2.0 ** 126
    out = torch.full_like(q, 9.0)
    assert cache.append(q, k, v, cu_of(new), vec(*order), layer=1, out=out) is out
    cache.check()
    assert torch.equal(out[:T], q[:T]) and bool((out[T:] == 9.0).all())
    assert torch.equal(cache.k[0], k0[0]) and torch.equal(cache.v[0], v0[0])
    for got, given in zip(ref.unpack(cache, 1), (k, v)):
        codes, s, z, bad = ref.quantise(given, bits, group)
        at = 0
        for b, n in enumerate(new):
            for i in range(n):
                pos = lens[b] - n + i
                p = int(cache.table[order[b], pos // page])
                assert torch.equal(got[0][p, pos % page][~bad[at].repeat_interleave(group, -1)],
                                   codes[at][~bad[at].repeat_interleave(group, -1)])
                assert same(got[1][p, pos % page], s[at]) and same(got[2][p, pos % page], z[at])
                at += 1
    # nothing else was written: the tokens that were there, the free pages
    live = torch.zeros(cache.k.shape[1], page, dtype=torch.bool)
    for b, n in enumerate(new):
        for i in range(lens[b] - n, lens[b]):
            live[int(cache.table[order[b], i // page]), i % page] = True
    chunks = -(-D * bits // 128)
    for now, before, is_v in ((cache.k[1].cpu(), k0[1].cpu(), False), (cache.v[1].cpu(), v0[1].cpu(), True)):
        c, c0 = (ref.tokens(t[..., :page * chunks * 16], page, chunks, bits, is_v).transpose(1, 2) for t in (now, before))
        p, p0 = (t[..., page * chunks * 16:].reshape(-1, HKV, page, 4 * (D // group)).transpose(1, 2) for t in (now, before))
        assert torch.equal(c[~live], c0[~live]) and torch.equal(p[~live], p0[~live])
        assert not bool(c[live][..., D * bits // 8:].any())  # columns that do not exist


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,bits,group,rot", [(128, 4, 64, 128), (128, 8, 128, 64), (80, 8, 80, 40), (64, 4, 64, 64), (96, 4, 96, 6)])
def test_append_turns_then_quantises(kv, dtype, layout, D, bits, group, rot):
    H, HKV, lens, new = 6, 2, [700, 90], [333, 1]
    cache, _ = ref.make(kv, lens, 16, HKV, D, bits, group, dtype, stored=False)
    rope = kv.Rope(D, rot, 500000.0, layout, dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192))
    q, k, v = (randn(334, h, D, dtype=dtype, seed=i) for i, h in enumerate((H, HKV, HKV)))
    got = cache.append(q, k, v, cu_of(new), rope=rope)
    cache.check()
    pos = torch.cat([torch.arange(n - a, n) for a, n in zip(new, lens)]).cuda()
    scaling = dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192)
    want, bound = _kv_ref.rotate(q, pos, rot, 500000.0, scaling, layout)
    _kv_ref.close(got, want, bound, "q")
    want, bound = (x.cpu() for x in _kv_ref.rotate(k, pos, rot, 500000.0, scaling, layout))
    at = 0
    for b, n in enumerate(new):
        (val, s, z, _), (vv, _, _, _) = ref.held(cache, b)
        x, e = want[at:at + n], bound[at:at + n]
        # half a step, the turn's error, and the three fp32 roundings of a code (of a quotient up to 255)
        assert bool(((val[-n:] - x).abs() <= s[-n:] * (0.5 + 255 * 3 * 2.0 ** -24) + e).all())
        # the scale is the range's, but for the roundings of offset and scale up to a bf16
        g = x.unflatten(-1, (-1, group))
        e = e.unflatten(-1, (-1, group)).amax(-1)
        most, least = g.amax(-1), g.amin(-1)
        step = (most - least + 2 * e + 2.0 ** -7 * (least.abs() + e)) / (2 ** bits - 1) * (1 + 2.0 ** -7)
        assert bool((s[-n:].unflatten(-1, (-1, group))[..., 0] <= step * (1 + 2.0 ** -20)).all())
        codes, vs, vz, _ = ref.quantise(v[at:at + n], bits, group)
        up = lambda t: t.double().repeat_interleave(group, -1)  # noqa: E731
        assert torch.equal(vv[-n:], up(vs) * codes.double() + up(vz))
        at += n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_strided_unaligned_and_in_place(kv, dtype):
    D, HKV, H = 64, 2, 4
    lens = [37, 70]
    rope = kv.Rope(D, 32, layout="half")
    packed = randn(107, H + 2 * HKV, D, dtype=dtype, seed=3)
    a, _ = ref.make(kv, lens, 16, HKV, D, 4, D, dtype, stored=False, poison=False)
    b, _ = ref.make(kv, lens, 16, HKV, D, 4, D, dtype, stored=False, poison=False)
    cu = cu_of(lens)
    q, k, v = packed[:, :H], packed[:, H:H + HKV], packed[:, H + HKV:]
    one = a.append(q, k, v, cu, rope=rope)
    wide = torch.zeros(107, (H + 2 * HKV) * D + 1, dtype=dtype, device="cuda")  # odd strides and addresses
    odd = wide[:, 1:].unflatten(1, (H + 2 * HKV, D))
    odd.copy_(packed)
    two = b.append(odd[:, :H], odd[:, H:H + HKV], odd[:, H + HKV:], cu, rope=rope)
    assert torch.equal(one, two) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    here = q.contiguous()
    assert b.append(here, k, v, cu, rope=rope, out=here) is here
    assert torch.equal(one, here) and torch.equal(a.k, b.k)
    # one token or one head of q, whatever its other stride; no q
    assert b.append(None, k, v, cu, rope=rope) is None and torch.equal(a.k, b.k)


# ---- read
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("D,bits,group", ref.SHAPES)
def test_read_gives_back_what_is_held(kv, out_dtype, D, bits, group):
    lens, page, HKV = [45, 0, 300, 16], 16, 2
    order = [2, 0, 4, 1]
    cache, _ = ref.make(kv, lens, page, HKV, D, bits, group, BF, planes=2, slots=5, order=order, shift=0.3)
    cases = [([45, 0, 300, 16], None), ([1, 0, 7, 16], None), ([20, 0, 33, 0], [25, 0, 77, 0])]
    for rows, first in cases:
        T, pad = sum(rows), 3
        out = [torch.full((T + pad, HKV, D), 7.0, dtype=out_dtype, device="cuda") for _ in range(2)]
        got = cache.read(cu_of(rows), T + pad, vec(*order), None if first is None else vec(*first), layer=1, out=out)
        cache.check()
        for x, which in zip(got, range(2)):
            want = []
            for b, n in enumerate(rows):
                at = lens[b] - n if first is None else first[b]
                want.append(ref.held(cache, order[b], 1)[which][0][at:at + n])
            assert torch.equal(x[:T].cpu(), torch.cat(want).float().to(out_dtype))
            assert bool((x[T:] == 7.0).all())
    k, v = cache.read(cu_of([3]), 3, vec(4))
    assert k.dtype == BF and k.shape == v.shape == (3, HKV, D)
    assert cache.read(cu_of([]), 0)[0].shape == (0, HKV, D)


def test_read_of_tokens_that_do_not_exist(kv):
    cache, _ = ref.make(kv, [20, 30], 8, 1, 32, 4, 32, BF, slots=3)
    cache.table[1, 2] = -1
    cu = cu_of([20, 30, 2, 4])
    k, v = cache.read(cu, 56, vec(0, 1, 9, 0), vec(0, 0, 0, 18))
    with pytest.raises(kv.CacheError) as e:
        cache.check()
    assert e.value.bits == kv.BAD_PAGE | kv.BAD_SLOT | kv.BAD_LENGTH
    for x, which in ((k, 0), (v, 1)):
        a, b = ref.held(cache, 0)[which][0], ref.held(cache, 1)[which][0]
        b[16:24] = 0.0
        want = torch.cat([a, b, torch.zeros(2, 1, 32, dtype=torch.float64), a[18:20], torch.zeros(2, 1, 32, dtype=torch.float64)])
        assert torch.equal(x.cpu(), want.to(BF))


# ---- attend
def check_attend(kv, dtype, new, lens, page, H, HKV, D, bits, group, causal=True, window=0, out_dtype=None, pad=0, seed=0,
                 scale=None, tiles=False, shift=0.0, slots=None):
    order = list(range(len(lens)))[::-1] if slots is None else slots
    cache, _ = ref.make(kv, lens, page, HKV, D, bits, group, dtype, seed=seed, planes=2, slots=max(order, default=0) + 1,
                        order=order, shift=shift)
    T = sum(new)
    q = randn(T + pad, H, D, dtype=dtype, seed=seed + 1, mul=1.5)
    if pad:
        q[T:] = math.nan
    odt = out_dtype or dtype
    out, lse = torch.full((T + pad, H, D), 7.0, dtype=odt, device="cuda"), torch.full((T + pad, H), 7.0, device="cuda")
    cache.attend(q, cu_of(new), vec(*order), scale, causal, window, layer=1, out=out, lse=lse)
    cache.check()
    want, want_l, bo, bl = ref.attend(cache, q[:T], new, order, D ** -0.5 if scale is None else scale, causal, window, 1, tiles,
                                      odt == F32)
    _kv_ref.close(out[:T].cpu(), want, bo, "O")
    seen = torch.isfinite(want_l)
    assert torch.equal(lse[:T].cpu() == -math.inf, ~seen)
    err = (lse[:T].cpu().double() - want_l)[seen].abs()
    assert bool((err <= bl[seen]).all()), float(err.max())
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
    # ... and as near as such arithmetic usually is, which is far inside the worst case: a bf16 output is its own rounding
    # (2^-8 / sqrt(12) of O's powers of two: 1.7e-3) and little more; probabilities of scores that are four times as
    # large as usual (scale 0.3) move four times as far with the rounding of tiles' K
    if T and bool(seen.any()):
        off = float((out[:T].cpu().double() - want).norm() / want.norm())
        assert off < (2.5e-3 if odt == BF else 2e-3 if tiles else 2e-6), off
    return cache, q, out, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,bits,group", ref.SHAPES)
def test_attend_decoding(kv, dtype, D, bits, group):
    check_attend(kv, dtype, [1, 1, 0, 1, 1], [1, 300, 40, 33, 64], 16, 8, 2, D, bits, group, shift=0.2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 128)])
@pytest.mark.parametrize("new,lens,page,H,HKV,kw", [
    ([5], [5], 8, 4, 4, {}),                                    # a prompt from its beginning
    ([3, 2, 1], [700, 2, 129], 32, 16, 2, {"window": 100}),
    ([4, 4], [2000, 31], 64, 4, 1, {"causal": False}),
    ([2, 1], [513, 512], 256, 5, 5, {"window": 1}),
    ([1, 3], [40, 50], 1024, 24, 3, {"pad": 5, "scale": 0.3}),
    ([7, 0, 2], [90, 0, 9], 16, 6, 2, {"causal": False, "window": 20, "pad": 2}),
    ([1] * 40, [1 + 37 * i for i in range(40)], 16, 4, 1, {}),
    ([6], [600], 16, 5, 1, {}),                                 # more rows than one pass over the keys takes, fewer than tiles
    ([4, 3], [333, 90], 64, 16, 2, {"window": 50}),
    ([1, 0, 0, 0, 0, 0, 0, 0], [70, 0, 3, 4, 5, 6, 7, 8], 8, 128, 1, {})])  # 128 heads to one of the cache
def test_attend_masks_and_shapes(kv, dtype, bits, group, new, lens, page, H, HKV, kw):
    check_attend(kv, dtype, new, lens, page, H, HKV, 128, bits, group, **kw)


@pytest.mark.parametrize("dtype,out_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("bits", [4, 8])
def test_attend_other_output_type(kv, dtype, out_dtype, bits):
    check_attend(kv, dtype, [1, 2], [900, 77], 16, 8, 2, 64, bits, 64, out_dtype=out_dtype)


@pytest.mark.parametrize("bits", [4, 8])
def test_attend_rows_that_see_nothing(kv, bits):
    cache, _ = ref.make(kv, [0, 5], 8, 1, 64, bits, 64, BF)
    q = randn(4, 2, 64, dtype=BF)
    # a sequence without tokens, and one whose window lies before its first: positions -1 .. see nothing
    cache.lens[1] = 1
    o, lse = cache.attend(q, cu_of([2, 2]))
    cache.lens[0] = 0
    assert bool((o[:3] == 0).all()) and bool((lse[:3] == -math.inf).all())
    assert bool(torch.isfinite(lse[3]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bits", [4, 8])
def test_attend_strided_queries_and_forked_slots(kv, dtype, bits):
    cache, _ = ref.make(kv, [333, 50], 16, 2, 64, bits, 64, dtype, slots=3)
    wide = randn(3, 12, 64, dtype=dtype, seed=5)
    a = cache.attend(wide[:, 2:10], cu_of([1, 2]))
    b = cache.attend(wide[:, 2:10].contiguous(), cu_of([1, 2]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a slot forked from one and the slot itself, in one batch: the same values, each within its bound
    cache.fork(vec(0), vec(2))
    q = wide[:1, 2:10].expand(2, -1, -1).contiguous()
    o, lse = cache.attend(q, cu_of([1, 1]), vec(0, 2))
    cache.check()
    want, want_l, bo, bl = ref.attend(cache, q, [1, 1], [0, 0], 64 ** -0.5, True, 0)
    _kv_ref.close(o.cpu(), want, bo, "O")
    assert bool(((lse.cpu().double() - want_l).abs() <= bl).all())


# ---- chunks of a prompt (tensor-core tiles)
@pytest.mark.parametrize("D,bits,group", ref.SHAPES)
def test_attend_chunks(kv, D, bits, group):
    check_attend(kv, BF, [70, 40, 0, 90], [70, 300, 20, 217], 16, 8, 2, D, bits, group, tiles=True, shift=0.2, pad=3)


@pytest.mark.parametrize("bits,group", [(4, 64), (8, 128), (4, 128)])
@pytest.mark.parametrize("new,lens,page,H,HKV,kw", [
    ([300], [300], 8, 4, 4, {}),
    ([129, 65], [1000, 65], 32, 16, 2, {"window": 100}),
    ([200, 64], [700, 131], 64, 4, 1, {"causal": False}),
    ([90, 17], [513, 512], 256, 5, 5, {"window": 1}),
    ([33, 31], [1040, 50], 1024, 24, 3, {"pad": 50, "scale": 0.3}),
    ([100, 0, 35], [190, 0, 35], 16, 6, 2, {"causal": False, "window": 20, "pad": 2}),
    ([150], [2000], 128, 7, 1, {"out_dtype": F32}),
    ([2, 1], [50, 1100], 1024, 128, 1, {}),                     # a tile to each token
    ([1], [77], 8, 96, 1, {"window": 60}),
    ([200], [200], 16, 100, 50, {"scale": 0.02})])
def test_attend_chunks_masks_and_shapes(kv, bits, group, new, lens, page, H, HKV, kw):
    check_attend(kv, BF, new, lens, page, H, HKV, 128, bits, group, tiles=True, **kw)
