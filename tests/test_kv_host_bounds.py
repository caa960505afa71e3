"""Host-only checks of include/fakv.h at the edges of its rules (no call here reaches a kernel)."""
import math

import pytest


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
