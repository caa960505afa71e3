"""Host-only checks of include/fakv.h at the edges of its rules (no call here reaches a kernel)."""
import ctypes
import math

import pytest

A = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    from attention_fa_fwd_02_gb300 import kv as m
    return m


@pytest.mark.parametrize("factor,want", [(0.01, 1.0), (0.5, 1.0), (1.0, 1.0), (4.0, 0.1 * math.log(4.0) + 1.0)])
def test_yarn_multiplies_by_one_where_nothing_is_stretched(kv, factor, want):
    r = kv.Rope(64, scaling=dict(kind="yarn", factor=factor, original=4096), device="cpu")
    assert abs(r.mscale - want) < 1e-6
    assert kv.Rope(64, scaling=dict(kind="yarn", factor=factor, original=4096, mscale=0.7), device="cpu").mscale == 0.7


@pytest.mark.parametrize("stride", [0, 5, -64, 1 << 60])
def test_the_plane_stride_of_one_plane_is_no_matter(kv, stride):
    c = kv.fakv_cache(K=A, V=A, table=A, lens=A, refs=A, plane_stride=stride, page_stride=2048, token_stride=128,
                      head_stride=64, table_stride=10, planes=1, num_pages=100, page_size=16, HKV=2, D=64, max_slots=4,
                      max_pages=10, dtype=1)
    t = kv.fakv_tokens(B=0, T=3, H=4, q_token=256, q_head=64, scale=0.1, causal=1, out_dtype=1)
    lib, C = kv._lib(), ctypes.byref(c)
    assert lib.fakv_attend(A, A, A, A, None, C, ctypes.byref(t), None) == 0  # (no sequences: nothing is enqueued)
    assert lib.fakv_append(A, A, A, A, A, None, None, C, ctypes.byref(t), None) == 0
    assert lib.fakv_grow(C, A, A, 0, None) == 0 and lib.fakv_fork(C, A, A, 0, None) == 0
    c.planes = 2
    assert lib.fakv_attend(A, A, A, A, None, C, ctypes.byref(t), None) in (1, 3)
