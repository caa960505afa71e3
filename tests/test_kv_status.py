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
