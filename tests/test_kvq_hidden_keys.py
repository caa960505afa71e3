"""Keys that a row's mask hides have no part in it, however large their K and V are: attention over the cache in 4 or 8 bits
with one token far larger than the others, seen by some of a call's rows and hidden from the rest, against bounds that
each row's own keys give (_kvq_seen.py)."""
import pytest
import torch

import _kv_ref
import _kvq_ref as ref
import _kvq_seen as seen

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
KINDS = [(BF, BF, 4), (BF, F32, 4), (F32, F32, 4), (F32, BF, 4), (BF, BF, 7), (BF, BF, 70), (BF, F32, 70)]  # q, O, rows


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_fa_fwd_02_gb300 import kv as m
    return m


def run(kv, dtype, out_dtype, rows, D, bits, group, which, factor, at, n, causal=True, window=0, H=4):
    """One sequence of n tokens, the last `rows` of them new; K or V of token `at` times `factor`."""
    cache, given = ref.make(kv, [n], 16, 1, D, bits, group, dtype, seed=3)
    k, v = (x.clone() for x in given[0])
    (k if which == "k" else v)[at] *= factor
    cache.append(None, k, v, torch.tensor([0, n], dtype=torch.int32).cuda())
    g = torch.Generator().manual_seed(8)
    q = torch.randn(rows, H, D, generator=g).to(dtype).cuda()
    o, l = cache.attend(q, torch.tensor([0, rows], dtype=torch.int32).cuda(), causal=causal, window=window, out_dtype=out_dtype)
    cache.check()
    tiles = dtype == BF and rows > 16
    want, want_l, bo, bl = seen.attend(cache, q, [rows], [0], D ** -0.5, causal, window, 0, tiles, out_dtype == F32)
    _kv_ref.close(o.cpu(), want, bo, "O")
    assert bool(((l.cpu().double() - want_l).abs() <= bl).all()), float((l.cpu().double() - want_l).abs().max())
    p, hidden = torch.arange(n - rows, n), torch.zeros(rows, dtype=torch.bool)
    if causal:
        hidden |= p < at
    if window:
        hidden |= at <= p - window
    assert bool(hidden.any()) and not bool(hidden.all())


@pytest.mark.parametrize("dtype,out_dtype,rows", KINDS)
@pytest.mark.parametrize("which", ["v", "k"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("factor", [2.0 ** 16, 2.0 ** 31, -2.0 ** 60])
def test_a_large_token_behind_a_row(kv, dtype, out_dtype, rows, which, bits, factor):
    """In the middle of the new tokens: hidden from the earlier ones of a causal call."""
    n = 200 + rows
    run(kv, dtype, out_dtype, rows, 128, bits, 64 if bits == 4 else 128, which, factor, n - rows // 2, n)


@pytest.mark.parametrize("dtype,out_dtype,rows", KINDS)
@pytest.mark.parametrize("which", ["v", "k"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("causal", [False, True])
def test_a_large_token_before_a_rows_window(kv, dtype, out_dtype, rows, which, bits, causal):
    """A token that the first rows' windows hold and the last rows' do not."""
    n = 300 + rows
    run(kv, dtype, out_dtype, rows, 64, bits, 64, which, 2.0 ** 45, n - 40 - rows // 2, n, causal, 40)


@pytest.mark.parametrize("dtype,out_dtype,rows", KINDS)
@pytest.mark.parametrize("bits", [4, 8])
def test_small_keys_beside_large_ones(kv, dtype, out_dtype, rows, bits):
    """K of very different sizes, all seen: the large ones' scores far below the others', so that these alone make O."""
    D, n, H = 64, 130 + rows, 2
    cache, given = ref.make(kv, [n], 16, 1, D, bits, D, dtype, seed=4, stored=False)
    g = torch.Generator().manual_seed(9)
    q = (1 + 0.3 * torch.randn(rows, H, D, generator=g)).to(dtype).cuda()
    k = torch.randn(n, 1, D, generator=g)
    k[5::7] = -(2.0 ** 20) * (1 + 0.2 * torch.rand(k[5::7].shape, generator=g))
    k[3::31] *= 2.0 ** -20
    v = torch.randn(n, 1, D, generator=g)
    cache.append(None, k.to(dtype).cuda(), v.to(dtype).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    o, l = cache.attend(q, torch.tensor([0, rows], dtype=torch.int32).cuda(), out_dtype=out_dtype)
    cache.check()
    want, want_l, bo, bl = seen.attend(cache, q, [rows], [0], D ** -0.5, True, 0, 0, dtype == BF and rows > 16, out_dtype == F32)
    _kv_ref.close(o.cpu(), want, bo, "O")
    assert bool(((l.cpu().double() - want_l).abs() <= bl).all()), float((l.cpu().double() - want_l).abs().max())
    assert float(want_l.abs().max()) < 50
