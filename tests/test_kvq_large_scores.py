"""Scores far beyond what a softmax tells apart, over the cache in 4 or 8 bits: K and q are finite, so O and LSE are, and a
row is its largest key's V. (A product that is fused with taking its row's reference off keeps bits that the reference has
been rounded from: of scores of 2^30 that is 2^6 and more, either way.)"""
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


@pytest.mark.parametrize("dtype,rows", [(BF, 1), (BF, 6), (F32, 3), (BF, 60)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("k,q", [(2.0 ** 12, 2.0 ** 9), (2.0 ** 20, 2.0 ** 10), (2.0 ** 70, 2.0 ** 30), (-(2.0 ** 20), 2.0 ** 60)])
def test_rows_of_large_scores(kv, dtype, rows, bits, k, q):
    D, n, H = 128, 500, 4
    cache, given = ref.make(kv, [n], 16, 1, D, bits, D, dtype, seed=5)
    cache.append(None, given[0][0] * k, given[0][1], torch.tensor([0, n], dtype=torch.int32).cuda())
    g = torch.Generator().manual_seed(6)
    x = (torch.randn(rows, H, D, generator=g) * q).to(dtype).cuda()
    for odt in (BF, F32):
        o, l = cache.attend(x, torch.tensor([0, rows], dtype=torch.int32).cuda(), out_dtype=odt)
        cache.check()
        assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(l).all())
        want, want_l, bo, bl = seen.attend(cache, x, [rows], [0], D ** -0.5, True, 0, 0, dtype == BF and rows > 16, odt == F32)
        _kv_ref.close(o.cpu(), want, bo, "O")
        assert bool(((l.cpu().double() - want_l).abs() <= bl).all())


@pytest.mark.parametrize("dtype,rows", [(BF, 1), (BF, 6), (F32, 3), (BF, 60)])
@pytest.mark.parametrize("bits", [4, 8])
def test_queries_far_below_one(kv, dtype, rows, bits):
    """q of 2^-90, as exact as any other, with K of 2^70 and a softmax scale of 2^20: ordinary scores."""
    D, n, H = 64, 300, 4
    cache, given = ref.make(kv, [n], 16, 1, D, bits, D, dtype, seed=7)
    cache.append(None, given[0][0] * 2.0 ** 70, given[0][1], torch.tensor([0, n], dtype=torch.int32).cuda())
    g = torch.Generator().manual_seed(8)
    q = (torch.randn(rows, H, D, generator=g) * 2.0 ** -90).to(dtype).cuda()
    scale = 2.0 ** 20 * D ** -0.5
    o, l = cache.attend(q, torch.tensor([0, rows], dtype=torch.int32).cuda(), scale=scale)
    cache.check()
    want, want_l, bo, bl = seen.attend(cache, q, [rows], [0], scale, True, 0, 0, dtype == BF and rows > 16)
    _kv_ref.close(o.cpu(), want, bo, "O")
    assert bool(((l.cpu().double() - want_l).abs() <= bl).all())
