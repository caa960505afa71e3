"""Outputs of a reading back of the cache in 4 or 8 bits that lie over each other are refused, on the host."""
import ctypes

import pytest

from test_kvq_host import A, cache, kv, tokens  # noqa: F401 (kv is a fixture)


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2)])
def test_outputs_that_overlap_are_refused(kv, dtype, size):  # noqa: F811
    lib, C, P = kv._lib(), ctypes.byref(cache(kv)), ctypes.byref(tokens(kv, out_dtype=dtype))
    rows = 3 * 2 * 128 * size  # T HKV D
    for k, v in ((A, A), (A, A + 16), (A + 16, A), (A, A + rows - 16), (A + rows - 16, A)):
        assert lib.fakv_qread(k, v, A, None, None, C, P, None) == 1
    # nothing to write
    assert lib.fakv_qread(A, A, A, None, None, C, ctypes.byref(tokens(kv, T=0, out_dtype=dtype)), None) == 0
