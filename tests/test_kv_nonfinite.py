"""GPU checks that what is not finite in a row of q, or in a page, reaches the outputs of the rows that see it, the
same whether a sequence is worked on whole or cut between workers, and no other row's."""
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


# new tokens, lengths: a short sequence (worked on whole) and a long one (cut); 300 tokens: the tensor-core tiles of bf16
@pytest.mark.parametrize("dtype,n", [(BF, 1), (BF, 4), (BF, 300), (F32, 1), (F32, 5), (F32, 40)])
@pytest.mark.parametrize("lens", [(310, 305), (9000, 305), (40000,)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_a_row_of_q(kv, dtype, n, lens, what):
    cache = ref.make_cache(kv, list(lens), 16, 2, 64, dtype)
    B, H = len(lens), 8
    g = torch.Generator().manual_seed(1)
    q = torch.randn(B * n, H, 64, generator=g).to(dtype).cuda()
    cu = cu_of([n] * B)
    want, want_l = cache.attend(q, cu, out_dtype=F32)
    _, _, bo, bl = ref.attend(cache, q, [n] * B, list(range(B)), 0.125, True, 0, one_term=dtype == BF)
    bo, bl = 2 * bo, 2 * bl  # between two results, each within its bound
    bad = torch.zeros(B * n, H, dtype=torch.bool, device="cuda")
    for t, h in {(0, 0), (n // 2, 5), (B * n - 1, H - 1)}:
        # (a column of both signs over the keys: inf and -inf scores, so NaN in the sums)
        q[t, h, 3] = float(what)
        bad[t, h] = True
    o, lse = cache.attend(q, cu, out_dtype=F32)
    cache.check()
    assert bool(torch.isnan(o[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    if what == "nan":
        assert torch.equal(o[~bad], want[~bad]) and torch.equal(lse[~bad], want_l[~bad])
    else:
        # (an infinite score moves the maxima of the rows beside it at another step: other roundings of the same sums)
        for x, y, slack in ((o, want, bo), (lse, want_l, bl)):
            ref.close(x[~bad], y[~bad].double(), slack[~bad], what)


@pytest.mark.parametrize("dtype,n", [(BF, 1), (BF, 64), (F32, 2)])
@pytest.mark.parametrize("size", [200, 30000])
def test_a_key(kv, dtype, n, size):
    # one key of one kv head of the first sequence: every query row of that head sees it
    cache = ref.make_cache(kv, [size, 500], 16, 2, 64, dtype)
    q = torch.randn(2 * n, 4, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    cu = cu_of([n, n])
    want, want_l = cache.attend(q, cu)
    p = size // 2
    cache.k[0, cache.table[0, p // 16].long(), p % 16, 1, 7] = float("nan")
    o, lse = cache.attend(q, cu)
    assert bool(torch.isnan(o[:n, 2:]).all()) and bool(torch.isnan(lse[:n, 2:]).all())
    for x, y in ((o, want), (lse, want_l)):
        assert torch.equal(x[:n, :2], y[:n, :2]) and torch.equal(x[n:], y[n:])
