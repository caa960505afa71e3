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


@pytest.mark.parametrize("kw", [dict(qo_token=0), dict(qo_head=0), dict(ko_token=0), dict(ko_head=32),
                                dict(qo_token=63), dict(T=1, qo_head=16), dict(H=1, qo_token=48)])
def test_rope_refuses_outputs_whose_rows_overlap(kv, kw):
    lib = kv._lib()

    def call(same=False, **kw):
        d = dict(T=3, H=4, HKV=2, D=64, dtype=1, positions_64=1, q_token=256, q_head=64, k_token=128, k_head=64,
                 qo_token=256, qo_head=64, ko_token=128, ko_head=64)
        d.update(kw)
        r = kv.fakv_rope(A, 64, 0, 1.0)
        if same:  # in place: the inputs' strides are the outputs'
            for x in ("q", "k"):
                for s in ("token", "head"):
                    d[f"{x}_{s}"] = d[f"{x}o_{s}"]
        b = 2 * A if not same else A
        return lib.fakv_rope_apply(A, A, b, b, A, ctypes.byref(r), ctypes.byref(kv.fakv_rope_params(**d)), None)

    assert call(**kw) == 1 and call(same=True, **kw) == 1
