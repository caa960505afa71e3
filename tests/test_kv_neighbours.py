"""GPU checks that a sequence's outputs do not change by a bit with rows that are not its own: those behind the last
sequence, another sequence's beside its own in a tile, or what an earlier call left in shared memory. (Lengths are the
same in each: they decide where the work is cut.)"""
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


def randn(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


FILLS = [0.0, 1.0, -500.0, float("inf"), float("nan"), "loud", "louder"]


@pytest.mark.parametrize("dtype,n,H,HKV,D", [(BF, 150, 8, 2, 64), (BF, 77, 6, 2, 128), (BF, 9, 4, 4, 64), (BF, 301, 5, 1, 32),
                                             (F32, 40, 8, 2, 64), (F32, 3, 4, 2, 128)])
def test_rows_behind_the_last_sequence(kv, dtype, n, H, HKV, D):
    cache = ref.make_cache(kv, [n + 9000], 16, HKV, D, dtype)
    pad = 200
    q = randn(n + pad, H, D, dtype=dtype, seed=1)
    got = []
    for fill in FILLS:
        q[n:] = randn(pad, H, D, dtype=dtype, seed=len(fill)) * (20 if fill == "loud" else 300) if isinstance(fill, str) else fill
        for odt in (BF, F32):
            got.append([x[:n].clone() for x in cache.attend(q, cu_of([n]), out_dtype=odt)])
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, got[i % 2][0]) and torch.equal(lse, got[i % 2][1]), FILLS[i // 2]


@pytest.mark.parametrize("H,HKV", [(8, 2), (6, 2), (5, 1), (7, 1)])
def test_a_neighbour_in_the_same_tile(kv, H, HKV):
    new = [50, 30, 121]
    cache = ref.make_cache(kv, [9000, 7000, 15000], 16, HKV, 64, BF)
    q = randn(sum(new), H, 64, dtype=BF, seed=2)
    want = cache.attend(q, cu_of(new))
    for mul in (0.0, 10.0, 200.0):
        x = q.clone()
        x[50:80] = randn(30, H, 64, dtype=BF, seed=9) * mul
        o, lse = cache.attend(x, cu_of(new))
        for a, b in ((o, want[0]), (lse, want[1])):
            assert torch.equal(a[:50], b[:50]) and torch.equal(a[80:], b[80:]), mul


@pytest.mark.parametrize("H,HKV", [(3, 1), (5, 1), (6, 2), (7, 1)])  # tiles of 126, 125, 126 and 126 rows of 128
def test_what_a_call_left_in_shared_memory(kv, H, HKV):
    cache = ref.make_cache(kv, [9000], 16, HKV, 64, BF)
    q, loud = randn(300, H, 64, dtype=BF, seed=3), randn(300, 8 * HKV, 64, dtype=BF, seed=4) * 300.0
    want = None
    for x in (torch.zeros_like(loud), loud, -loud, loud * 0.03):
        for _ in range(3):
            cache.attend(x, cu_of([300]))  # (whole tiles of 128 rows)
            got = cache.attend(q, cu_of([300]))
            want = want or [y.clone() for y in got]
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
