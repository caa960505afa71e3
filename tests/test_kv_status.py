"""GPU checks of PagedCache.check and of calls on streams of their own."""
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


def test_check_tells_of_a_wait_that_ran_out(kv):
    from attention_fa_fwd_02_gb300 import fa
    cache = ref.make_cache(kv, [10], 16, 1, 64, BF)
    cache.check()
    stream = torch.cuda.current_stream()
    roles = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert fa.fa_selftest_timeout(20_000_000, roles.data_ptr(), int(stream.cuda_stream)) == 0  # 20 ms
    with pytest.raises(fa.FAError) as e:
        cache.check()
    assert e.value.code == 5
    cache.check()  # read and cleared
    # both: the entries first, and the wait is not forgotten
    assert fa.fa_selftest_timeout(20_000_000, roles.data_ptr(), int(stream.cuda_stream)) == 0
    cache.grow(vec(7), vec(1))
    with pytest.raises(kv.CacheError):
        cache.check()
    with pytest.raises(fa.FAError):
        cache.check()
    cache.check()


def test_check_waits_for_every_stream(kv):
    cache = ref.make_cache(kv, [10], 16, 1, 64, BF)
    slots, add = vec(7), vec(1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    cache.grow(slots, add, stream=s)
    with pytest.raises(kv.CacheError):
        cache.check()
    cache.check()


def test_inputs_dropped_while_another_stream_reads_them(kv):
    """A tensor given to a call on another stream and dropped is not handed out again before the call has read it."""
    cache = ref.make_cache(kv, [100, 900], 16, 2, 64, BF)
    rope = kv.Rope(64)
    cu, pos = vec(0, 3, 6), torch.arange(6).cuda()
    keep = torch.randn(6, 8, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    want, want_l = cache.attend(keep, cu)
    want_r = rope.apply(keep, None, pos)[0]
    s = torch.cuda.Stream()
    for call, expect in ((lambda x: cache.attend(x, cu, stream=s)[0], want),
                         (lambda x: rope.apply(x, None, pos, stream=s)[0], want_r),
                         (lambda x: cache.append(x, x[:, :2], x[:, 2:4], cu, stream=s), keep)):
        q = keep.clone()
        address = q.data_ptr()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)
        got = call(q)
        del q
        other = [torch.full_like(keep, 9.0) for _ in range(20)]  # on the current stream, at once
        torch.cuda.current_stream().wait_stream(s)
        assert all(x.data_ptr() != address for x in other)
        assert torch.equal(got, expect)


def test_a_cache_dropped_while_another_stream_reads_it(kv):
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    cu, s = vec(0, 1), torch.cuda.Stream()
    cache = ref.make_cache(kv, [900], 16, 2, 64, BF)
    want = cache.attend(q, cu)[0]
    addresses, shape = {cache.k.data_ptr(), cache.v.data_ptr()}, cache.k.shape
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = cache.attend(q, cu, stream=s)[0]
    del cache
    other = [torch.full(shape, 9.0, dtype=BF, device="cuda") for _ in range(8)]
    torch.cuda.current_stream().wait_stream(s)
    assert not addresses & {x.data_ptr() for x in other}
    assert torch.equal(got, want)
