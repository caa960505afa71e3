"""Chunks over the cache in 4 or 8 bits with rows that see no key: sequences without tokens, new tokens that a length does not
count, and so come before the first one. They get O = 0 and LSE = -infinity, whatever the tile's other rows see."""
import math

import pytest
import torch

import _kv_ref
import _kvq_ref as ref
import _kvq_seen as seen

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_fa_fwd_02_gb300 import kv as m
    return m


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 25), (False, 0), (False, 25)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_no_key(kv, bits, causal, window, out_dtype, D):
    # new tokens, and how many of them (and of those before) the length counts
    new, lens = [150, 90, 0, 140, 70, 33], [150, 0, 40, 61, 300, 1]
    H, HKV = 4, 1
    cache, _ = ref.make(kv, lens, 16, HKV, D, bits, 64, BF, seed=2)
    g = torch.Generator().manual_seed(3)
    T = sum(new)
    q = torch.randn(T + 3, H, D, generator=g).to(BF).cuda()
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    out, lse = torch.full((T + 3, H, D), 7.0, dtype=out_dtype, device="cuda"), torch.full((T + 3, H), 7.0, device="cuda")
    cache.attend(q, cu, causal=causal, window=window, out=out, lse=lse)
    cache.check()
    want, want_l, bo, bl = seen.attend(cache, q[:T], new, list(range(6)), D ** -0.5, causal, window, 0, True, out_dtype == F32)
    nothing = want_l == -math.inf
    # 90 of a sequence without tokens; of 140 the first 79, of 33 the first 32, which come before every token
    assert int(nothing.sum()) == H * (90 + (79 + 32 if causal else 0))
    assert torch.equal(lse[:T].cpu() == -math.inf, nothing)
    assert bool((out[:T].cpu()[nothing] == 0).all())
    _kv_ref.close(out[:T].cpu(), want, bo, "O")
    err = (lse[:T].cpu().double() - want_l)[~nothing].abs()
    assert bool((err <= bl[~nothing]).all())
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
